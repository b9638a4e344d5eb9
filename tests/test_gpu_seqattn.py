"""Sequence attention (sliding window with sink tokens), forward and backward,
against the 64-bit reference within derived bounds, at the sizes and masks where
it can go wrong."""
import pytest
import torch

import seq_reference as ref
from shifted_window_attention_pad_b200 import binding as sb

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


def make(B, S, H, K, hd, dtype, seed=0, fused=False):
    gen = torch.Generator("cuda").manual_seed(seed)
    new = lambda n: torch.randn(B, S, n, hd, generator=gen, device="cuda").to(DT[dtype])
    if fused:
        x = new(H + 2 * K)
        return x[:, :, :H], x[:, :, H:H + K], x[:, :, H + K:], new(H)
    return new(H), new(K), new(K), new(H)


def run(q, k, v, g, window, sinks, lengths=None, flags=0, ws=None):
    d = sb.seq_desc_for(q, k, window=window, sinks=sinks, flags=flags)
    ws = sb.new_seq_workspace(d) if ws is None else ws
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = sb.seq_forward(d, q, k, v, lengths=n, want_lse=True, workspace=ws)
    dq, dk, dv = sb.seq_backward(d, q, k, v, out, lse, g, lengths=n, workspace=ws)
    torch.cuda.synchronize()
    assert sb.swin_wattn_poll_status(ws) == 0
    return {"o": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


ALL = ("o", "lse", "dq", "dk", "dv")

# B, S, heads, kv_heads, hd, window, sinks, lengths, fused
CASES = [
    (1, 1, 1, 1, 64, 0, 0, None, False),
    (2, 1, 4, 2, 128, 1, 1, None, False),
    (2, 3, 2, 2, 32, 0, 0, None, True),
    (1, 127, 2, 1, 64, 0, 0, None, False),
    (1, 128, 2, 2, 128, 0, 0, None, True),
    (1, 129, 3, 1, 64, 128, 0, None, False),
    (2, 300, 4, 2, 64, 1, 0, None, False),          # each token sees itself alone
    (2, 300, 4, 2, 128, 1, 3, None, True),
    (3, 257, 4, 4, 64, 40, 5, [257, 0, 1], False),  # a whole, an empty and a one-token sequence
    (2, 640, 8, 1, 128, 100, 130, [640, 511], False),   # sinks end inside the second tile
    (1, 1000, 2, 2, 64, 127, 7, None, True),
    (1, 1500, 2, 1, 128, 256, 1, [1300], False),
    (2, 2049, 2, 1, 64, 600, 4, [2049, 1025], False),   # sink tile in several query chunks
    (1, 2305, 1, 1, 128, 64, 200, None, False),         # two sink tiles in chunks
    (1, 1100, 8, 2, 64, 0, 9, None, False),
    (1, 700, 2, 1, 64, 64, 660, None, False),           # more sinks than windows
    (2, 200, 4, 2, 80, 50, 3, [200, 150], True),        # heads that do not fill a kernel's
    (1, 150, 2, 2, 8, 0, 0, None, False),
    (1, 130, 2, 1, 256, 33, 2, None, True),
    (2, 90, 2, 2, 136, 20, 0, [90, 64], False),
    # enough heads for pairs of query tiles (and more items than SMs): lengths that end
    # in either tile of a pair, windows and sinks whose key tiles only one tile needs
    (2, 1100, 40, 10, 64, 0, 0, [1100, 769], False),
    (2, 1100, 40, 40, 128, 200, 4, [1029, 896], False),
    (3, 700, 32, 4, 64, 130, 70, [700, 513, 257], True),
    (3, 700, 32, 32, 128, 64, 1, [640, 0, 129], False),
    (5, 515, 32, 8, 32, 300, 0, [515, 385, 1, 256, 255], False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:7]))
def test_against_the_reference(case, dtype):
    B, S, H, K, hd, window, sinks, lengths, fused = case
    q, k, v, g = make(B, S, H, K, hd, dtype, seed=S, fused=fused)
    got = run(q, k, v, g, window, sinks, lengths)
    want = ref.attention(q, k, v, window, sinks, lengths, g)
    ref.check(got, want, ALL)
    if lengths:   # padding is written as zeros
        for b, n in enumerate(lengths):
            for name in ALL:
                assert not got[name][b, n:].any(), name


@pytest.mark.parametrize("hd", [8, 40, 64, 72, 128])
def test_both_kernel_families_agree_with_the_reference(hd):
    q, k, v, g = make(1, 500, 4, 2, hd, "bf16", seed=3)
    want = ref.attention(q, k, v, 200, 4, None, g)
    for flags in (0, sb.SWIN_FLAG_FORCE_GENERIC):
        ref.check(run(q, k, v, g, 200, 4, flags=flags), want, ALL)


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("bf16", 128), ("f32", 64), ("bf16", 80), ("bf16", 192)])
def test_large_logits_and_equal_logits(dtype, hd):
    """A running maximum that keeps rising, and rows of equal logits."""
    q, k, v, g = make(1, 400, 2, 2, hd, dtype, seed=5)
    rise = torch.linspace(0.1, 12.0, 400, device="cuda")[None, :, None, None]
    k1 = (k.float() * rise).to(k.dtype)
    ref.check(run(q, k1, v, g, 0, 0), ref.attention(q, k1, v, 0, 0, None, g), ALL)
    zero = torch.zeros_like(q)
    got = run(zero, k, v, g, 150, 2)
    ref.check(got, ref.attention(zero, k, v, 150, 2, None, g), ALL)


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("bf16", 128), ("f32", 64), ("bf16", 80), ("bf16", 192)])
def test_padding_may_hold_anything(dtype, hd):
    q, k, v, g = make(2, 333, 4, 2, hd, dtype, seed=7)
    lengths = [333, 150]
    want = ref.attention(q, k, v, 90, 3, lengths, g)
    for t, x in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (g, float("-inf"))):
        t[1, 150:] = x
    got = run(q, k, v, g, 90, 3, lengths)
    ref.check(got, want, ALL)


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("bf16", 128), ("f32", 64), ("bf16", 80), ("bf16", 192)])
def test_a_nan_reaches_only_the_rows_that_see_it(dtype, hd):
    """Token 200 of sequence 0 holds NaN: rows that do not see it keep their
    results, those that do are NaN."""
    S, window, sinks, t = 420, 60, 2, 200
    q, k, v, g = make(1, S, 2, 1, hd, dtype, seed=9)
    want = ref.attention(q, k, v, window, sinks, None, g)
    sees = ref.visible(S, S, window, sinks, "cuda")[:, t]          # queries that see key t
    seen = ref.visible(S, S, window, sinks, "cuda")[t]             # keys that query t sees
    clean = lambda x, ok: {n: x[n][:, ok] for n in x}
    cut = lambda w, ok: {n: (w[n][0][:, ok], w[n][1][:, ok]) for n in w}
    for which in ("v", "k"):
        bad = {"k": k.clone(), "v": v.clone()}
        bad[which][:, t] = float("nan")
        got = run(q, bad["k"], bad["v"], g, window, sinks)
        assert torch.isnan(got["o"][:, sees]).all()
        ref.check(clean(got, ~sees), cut(want, ~sees), ("o", "lse", "dq"))
    # a NaN gradient of query t spoils dq of t and dk, dv of the keys it sees
    g2 = g.clone()
    g2[:, t] = float("nan")
    got = run(q, k, v, g2, window, sinks)
    ref.check(got, want, ("o", "lse"))
    assert torch.isnan(got["dv"][:, seen]).all() and torch.isnan(got["dq"][:, t]).all()
    ref.check(clean(got, ~seen), cut(want, ~seen), ("dk", "dv"))
    others = torch.arange(S, device="cuda") != t
    ref.check(clean(got, others), cut(want, others), ("dq",))


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("which", ["q", "k", "v", "g", "all"])
def test_tensors_of_nan(which, dtype, hd):
    """A whole tensor of NaN (a run that has diverged): every row that sees one is
    NaN, and the call ends with its status in order."""
    t = dict(zip("qkvg", make(2, 700, 8, 4, hd, dtype, seed=31)))
    for name in t:
        if which in (name, "all"):
            t[name].fill_(NAN)
    got = run(t["q"], t["k"], t["v"], t["g"], 300, 2, [700, 401])
    for b, n in enumerate((700, 401)):
        for name in ("dq", "dk", "dv"):
            # dO does not meet V or Q in dV, P does not meet V
            if not (name == "dv" and which == "v"):
                assert torch.isnan(got[name][b, :n]).all(), name
            assert not got[name][b, n:].any(), name
        assert torch.isnan(got["o"][b, :n]).all() == (which != "g")
        assert torch.isfinite(got["o"][b, :n]).all() == (which == "g")


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("f32", 64)])
def test_lengths_out_of_range_count_as_the_bounds(dtype, hd):
    q, k, v, g = make(2, 140, 2, 2, hd, dtype, seed=11)
    got = run(q, k, v, g, 30, 1, [-5, 1000])
    ref.check(got, ref.attention(q, k, v, 30, 1, [0, 140], g), ALL)


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_repeated_calls_give_identical_bits(dtype, hd):
    q, k, v, g = make(2, 1300, 4, 1, hd, dtype, seed=13)
    a, b = (run(q, k, v, g, 200, 4, [1300, 700]) for _ in range(2))
    for name in ALL:
        assert torch.equal(a[name], b[name]), name


def test_small_differences_of_the_loss_match_the_gradients():
    """Directional central differences of sum(out * dout) in fp32: the
    difference of two sums of N = 2 * 70 * 4 * 64 terms of size about 1, each off
    by at most 2^-20, divided by the step."""
    q, k, v, g = make(2, 70, 4, 2, 64, "f32", seed=17)
    got = run(q, k, v, g, 20, 2)
    step = 2.0 ** -7
    d = sb.seq_desc_for(q, k, window=20, sinks=2)
    loss = lambda *x: (sb.seq_forward(d, *x).double() * g.double()).sum()
    for x, name in ((0, "dq"), (1, "dk"), (2, "dv")):
        e = torch.randn_like((q, k, v)[x])
        side = [loss(*[t + s * e if y == x else t for y, t in enumerate((q, k, v))])
                for s in (step, -step)]
        slope = float(side[0] - side[1]) / (2 * step)
        want = float((got[name].double() * e.double()).sum())
        # third-order term: |e| ~ 1 per element moves logits by at most a few step
        assert abs(slope - want) < 2e-2 * (1 + float((got[name].double() * e.double()).norm())), name


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("f32", 64)])
def test_captured_calls_follow_new_inputs_and_share_a_workspace(dtype, hd):
    q, k, v, g = make(2, 300, 4, 2, hd, dtype, seed=19)
    d = sb.seq_desc_for(q, k, window=70, sinks=3)
    ws = sb.new_seq_workspace(d)
    n = torch.tensor([300, 200], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 300, 4, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    f, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(f):
        sb.swin_seqattn_fwd(d, q, k, v, n, out, lse, ws)
    with torch.cuda.graph(b):
        sb.swin_seqattn_bwd(d, q, k, v, n, out, lse, g, dq, dk, dv, ws)
    for seed, lengths in ((21, [300, 200]), (22, [17, 299])):
        for dst, src in zip((q, k, v, g), make(2, 300, 4, 2, hd, dtype, seed=seed)):
            dst.copy_(src)
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        f.replay()
        b.replay()
        torch.cuda.synchronize()
        got = {"o": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
        ref.check(got, ref.attention(q, k, v, 70, 3, lengths, g), ALL)


def test_two_streams_with_a_workspace_each():
    q, k, v, g = make(1, 900, 4, 2, 64, "bf16", seed=23)
    one = run(q, k, v, g, 100, 2)
    d = sb.seq_desc_for(q, k, window=100, sinks=2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            ws = sb.new_seq_workspace(d)
            o, lse = sb.seq_forward(d, q, k, v, want_lse=True, workspace=ws)
            outs.append((o, lse, *sb.seq_backward(d, q, k, v, o, lse, g, workspace=ws)))
    torch.cuda.synchronize()
    for got in outs:
        for x, name in zip(got, ALL):
            assert torch.equal(x, one[name]), name


def test_own_workspaces_belong_to_the_stream(monkeypatch):
    """A call with a stream and no workspace takes its workspace on that stream:
    on the current one its memory could be handed on while the call runs."""
    q, k, v, g = make(1, 300, 4, 2, 64, "bf16", seed=29)
    one = run(q, k, v, g, 100, 2)
    d = sb.seq_desc_for(q, k, window=100, sinks=2)
    s, on = torch.cuda.Stream(), []
    empty = torch.empty

    def recorded(*a, **kw):
        on.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)

    out, lse = torch.empty_like(q), torch.empty_like(one["lse"])
    grads = [torch.empty_like(t) for t in (q, k, v)]
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", recorded)
    sb.swin_seqattn_fwd(d, q, k, v, None, out, lse, stream=s)
    sb.swin_seqattn_bwd(d, q, k, v, None, out, lse, g, *grads, stream=s)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert on == [s.cuda_stream] * 2
    for x, name in zip((out, lse, *grads), ALL):
        assert torch.equal(x, one[name]), name


def test_timeouts_are_reported():
    """The kernels' bounded wait: a barrier that nothing arrives on ends the call
    with a status, and the workspace serves the next call."""
    q, k, v, g = make(1, 200, 2, 2, 64, "bf16", seed=25)
    d = sb.seq_desc_for(q, k, window=0, flags=sb.SWIN_FLAG_TEST_TIMEOUT)
    ws = sb.new_seq_workspace(d)
    out, lse = sb.seq_forward(d, q, k, v, want_lse=True, workspace=ws)
    assert sb.swin_wattn_poll_status(ws) == sb.SWIN_ERR_TIMEOUT
    assert sb.swin_wattn_poll_status(ws) == 0
    sb.seq_backward(d, q, k, v, out.zero_(), lse.zero_(), g, workspace=ws)
    assert sb.swin_wattn_poll_status(ws) == sb.SWIN_ERR_TIMEOUT
    ref.check(run(q, k, v, g, 0, 0, ws=ws), ref.attention(q, k, v, 0, 0, None, g), ALL)


def test_wrappers_refuse_what_the_description_does_not_say():
    q, k, v, g = make(1, 40, 4, 2, 64, "bf16")
    d = sb.seq_desc_for(q, k, window=0)
    with pytest.raises(ValueError, match="shape"):
        sb.seq_forward(d, q[:, :39], k, v)
    with pytest.raises(ValueError, match="torch.bfloat16"):
        sb.seq_forward(d, q.float(), k, v)
    with pytest.raises(ValueError, match="strides"):
        sb.seq_forward(d, q, make(1, 40, 4, 2, 64, "bf16", fused=True)[1], v)
    with pytest.raises(ValueError, match="int32"):
        sb.seq_forward(d, q, k, v, lengths=torch.tensor([4], device="cuda"))
    with pytest.raises(sb.SwinWattnError):
        sb.seq_forward(d, q, k, v, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("hd", [64, 128])
def test_long_ragged_sequences_with_pairs_of_tiles(hd):
    """Rounds of every ring many times over, lengths that leave the second tile of a
    pair empty; sampled rows against the reference."""
    S, H, window, sinks, lengths = 4096, 16, 512, 4, [3501, 1799, 2]
    q, k, v, g = make(3, S, H, 4, hd, "bf16", seed=29)
    got = run(q, k, v, g, window, sinks, lengths)
    for b, n in enumerate(lengths):
        for name in ALL:
            assert not got[name][b, n:].any(), name
        for h in (0, 5):
            pick = lambda t, c: t[b:b + 1, :, c:c + 1]
            want = ref.attention(pick(q, h), pick(k, h // 4), pick(v, h // 4), window, sinks, [n],
                                 pick(g, h))
            ref.check({x: got[x][b:b + 1, :, h:h + 1] for x in ("o", "lse", "dq")}, want,
                      ("o", "lse", "dq"))
        heads = range(4, 8)   # of kv head 1
        parts = [ref.attention(pick(q, h), pick(k, 1), pick(v, 1), window, sinks, [n], pick(g, h))
                 for h in heads]
        for name in ("dk", "dv"):
            ref_sum = sum(w[name][0] for w in parts)
            bound = sum(w[name][1] for w in parts)
            ref.check({name: got[name][b:b + 1, :, 1:2]}, {name: (ref_sum, bound)}, (name,))


def test_one_row_sequences_in_a_large_batch():
    """More rows than 2^16 sequences."""
    q, k, v, g = make(70000, 2, 1, 1, 64, "bf16", seed=27)
    got = run(q, k, v, g, 0, 0)
    pick = torch.tensor([0, 1, 32767, 65535, 65536, 69999], device="cuda")
    want = ref.attention(q[pick], k[pick], v[pick], 0, 0, None, g[pick])
    ref.check({n: x[pick] for n, x in got.items()}, want, ALL)

"""The paged key-value cache: append, attention of one token, eviction, and a run
of them together, against the 64-bit reference."""
import pytest
import torch

import seq_reference as ref
from shifted_window_attention_pad_b200 import binding as sb

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


class Cache:
    """A pool of pages with shuffled tables; every row no token owns is NaN."""

    def __init__(self, B, H, K, hd, ps, mp, dtype, lengths, seed=0, tables=1, spare=3, **kw):
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.B, self.H, self.K, self.hd, self.ps, self.mp = B, H, K, hd, ps, mp
        self.dt = DT[dtype]
        pages = tables * B * mp + spare
        perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
        self.table = perm[:B * mp].reshape(B, mp).contiguous().cuda()
        self.dst = perm[B * mp:2 * B * mp].reshape(B, mp).contiguous().cuda() if tables > 1 else None
        self.k, self.v = (torch.full((pages, K, ps, hd), NAN, dtype=self.dt, device="cuda")
                          for _ in range(2))
        at = torch.arange(mp * ps, device="cuda")
        for b, n in enumerate(lengths):
            page, row = self.table[b].long()[at[:n] // ps], at[:n] % ps
            self.k[page, :, row], self.v[page, :, row] = self.new(n, K), self.new(n, K)
        self.set_lengths(lengths)
        self.desc = sb.make_cache_desc(B, H, hd, ps, pages, mp, dtype, kv_heads=K, **kw)
        self.ws = sb.new_cache_workspace(self.desc)

    def set_lengths(self, lengths):
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")

    def new(self, *shape):
        return torch.randn(*shape, self.hd, generator=self.gen, device="cuda").to(self.dt)

    def status(self):
        return sb.swin_wattn_poll_status(self.ws)

    def put(self, k_new, v_new):
        """The reference's own writing of a token per sequence."""
        k, v = self.k.clone(), self.v.clone()
        for b, n in enumerate(self.lengths.tolist()):
            if n:
                page, row = ref.row_of(self.table, b, n - 1, self.ps)
                k[page, :, row], v[page, :, row] = k_new[b], v_new[b]
        return k, v


def finite(got, want, names):
    """ref.check for results whose empty sequences are -inf in lse."""
    for name in names:
        x, (r, bound) = got[name].double(), want[name]
        gone = torch.isinf(r)
        assert torch.equal(x[gone], r[gone]), name
        over = (x[~gone] - r[~gone]).abs() - bound[~gone] - 1e-30
        assert over.numel() == 0 or float(over.max()) <= 0, (name, float(over.max()))


def same(a, b):
    """Equal bits (NaN of stale rows included)."""
    view = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.view(view), b.view(view))


# H, K, hd, page, max_pages, lengths, window, sinks
DECODE = [
    (1, 1, 64, 16, 2, [1], 0, 0),
    (8, 8, 64, 16, 20, [1, 2, 15, 16, 17, 300], 0, 0),
    (8, 2, 128, 12, 60, [700, 33, 0, 128, 129], 0, 0),         # page size 12, an empty sequence
    (16, 1, 128, 16, 80, [1200, 5], 0, 0),                     # 16 query heads of one kv head
    (24, 1, 64, 1, 260, [257, 31], 0, 0),                      # one-token pages, two head chunks
    (12, 2, 32, 64, 9, [513, 64, 65], 100, 0),
    (4, 4, 128, 32, 40, [1100, 3, 40], 37, 5),                 # window and sinks
    (4, 2, 64, 100, 7, [650, 651], 500, 200),                  # sinks and window meet
    (4, 2, 64, 16, 20, [300, 20], 1, 0),                       # the new token alone
    (8, 1, 64, 128, 64, [8192, 8000, 1], 0, 0),
    (6, 2, 80, 16, 30, [400, 77], 0, 0),                       # portable head sizes
    (5, 1, 256, 16, 10, [150, 1], 50, 2),
    (2, 2, 8, 4, 30, [99, 0], 0, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [True, False], ids=["new", "held"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(str(x) for x in c[:5]))
def test_decode_against_the_reference(case, new, dtype):
    H, K, hd, ps, mp, lengths, window, sinks = case
    B = len(lengths)
    c = Cache(B, H, K, hd, ps, mp, dtype, lengths, seed=H + hd, window=window, sinks=sinks,
              weights=True)
    q, kn, vn = c.new(B, H), c.new(B, K), c.new(B, K)
    w = torch.rand(B, K, mp * ps, generator=c.gen, device="cuda")
    nw = torch.full_like(w, 7.0)
    k_ref, v_ref = c.put(kn, vn) if new else (c.k.clone(), c.v.clone())
    out, lse = sb.cache_decode(c.desc, q, c.lengths, c.table, c.k, c.v,
                               k_new=kn if new else None, v_new=vn if new else None, weights=w,
                               new_weights=nw, want_lse=True, workspace=c.ws)
    assert c.status() == 0
    assert same(c.k, k_ref) and same(c.v, v_ref)      # the new row and no other
    want = ref.decode(q, k_ref, v_ref, c.table, lengths, ps, window, sinks, w)
    for b, n in enumerate(lengths):
        assert (nw[b, :, n:] == 7.0).all()            # nothing behind the sequence
        want["weights"][0][b, :, n:] = 7.0
    finite({"o": out, "lse": lse, "weights": nw}, want, ("o", "lse", "weights"))
    for b, n in enumerate(lengths):
        if n == 0:
            assert not out[b].any()
    # without weights: the same bits; in place: the same weights
    again = sb.cache_decode(c.desc, q, c.lengths, c.table, c.k, c.v, workspace=c.ws)
    assert same(again, out)
    w2 = w.clone()
    sb.cache_decode(c.desc, q, c.lengths, c.table, c.k, c.v, weights=w2, workspace=c.ws)
    for b, n in enumerate(lengths):
        assert torch.equal(w2[b, :, :n], nw[b, :, :n]) and torch.equal(w2[b, :, n:], w[b, :, n:])


def test_decode_of_many_ragged_sequences():
    lengths = [(37 * b * b) % 900 for b in range(150)]
    c = Cache(150, 4, 2, 64, 16, 60, "bf16", lengths, seed=2)
    q = c.new(150, 4)
    out, lse = sb.cache_decode(c.desc, q, c.lengths, c.table, c.k, c.v, want_lse=True,
                               workspace=c.ws)
    want = ref.decode(q, c.k, c.v, c.table, lengths, 16, 0, 0)
    finite({"o": out, "lse": lse}, want, ("o", "lse"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_of_a_batch_of_thousands(dtype):
    """More sequences than a block adds up itself, most of them short."""
    B = 2500
    lengths = [(b * 7919) % 40 if b % 100 else 150 + b // 10 for b in range(B)]
    c = Cache(B, 2, 1, 64, 16, 26, dtype, lengths, seed=3, weights=True)
    q = c.new(B, 2)
    w = torch.rand(B, 1, 26 * 16, generator=c.gen, device="cuda")
    nw = w.clone()
    out, lse = sb.cache_decode(c.desc, q, c.lengths, c.table, c.k, c.v, weights=w, new_weights=nw,
                               want_lse=True, workspace=c.ws)
    assert c.status() == 0
    pick = [0, 1, 2, 99, 100, 1023, 1024, 1025, 2300, 2400, 2499]
    at = torch.tensor(pick, device="cuda")
    want = ref.decode(q[at], c.k, c.v, c.table[at], [lengths[b] for b in pick], 16, 0, 0, w[at])
    finite({"o": out[at], "lse": lse[at], "weights": nw[at]}, want, ("o", "lse", "weights"))


def test_decode_takes_parts_of_one_projection():
    lengths = [200, 90]
    c = Cache(2, 8, 2, 64, 16, 20, "bf16", lengths, seed=4, q_stride=12 * 64, kv_stride=12 * 64)
    x = c.new(2, 12)
    k_ref, v_ref = c.put(x[:, 8:10], x[:, 10:])
    out = sb.cache_decode(c.desc, x[:, :8], c.lengths, c.table, c.k, c.v, k_new=x[:, 8:10],
                          v_new=x[:, 10:], workspace=c.ws)
    want = ref.decode(x[:, :8], k_ref, v_ref, c.table, lengths, 16, 0, 0)
    finite({"o": out}, want, ("o",))


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("f32", 64)])
def test_bad_pages_are_skipped_and_reported(dtype, hd):
    """Ids outside the pool are not followed: their positions do not count."""
    lengths = [100, 100, 20]
    c = Cache(3, 4, 2, hd, 16, 10, dtype, lengths, seed=6)
    q = c.new(3, 4)
    bad = c.table.clone()
    bad[0, 2], bad[0, 3] = -1, c.desc.num_pages      # positions 32 .. 63
    bad[2, :2] = 1 << 30                             # all of them
    out, lse = sb.cache_decode(c.desc, q, c.lengths, bad, c.k, c.v, want_lse=True, workspace=c.ws)
    assert c.status() == -1 and c.status() == 0
    left = [p for p in range(100) if not 32 <= p < 64]
    for h in range(4):
        kk = ref.gather(c.k, c.table.cpu(), 0, h // 2, left, 16).double()
        vv = ref.gather(c.v, c.table.cpu(), 0, h // 2, left, 16).double()
        p = torch.softmax(q[0, h].double() @ kk.T / hd ** 0.5, 0)
        # P and the output are rounded to the type, as in the reference's bounds
        u = ref.U[q.dtype] + 2e-6
        assert ((out[0, h].double() - p @ vv).abs() <= u * (p @ vv).abs() + u * (p @ vv.abs())).all()
    assert not out[2].any() and torch.isinf(lse[2]).all()
    # entries behind the last page are never read
    tail = c.table.clone()
    tail[0, 7:], tail[2, 2:] = -7, 1 << 30
    sb.cache_decode(c.desc, q, c.lengths, tail, c.k, c.v, workspace=c.ws)
    assert c.status() == 0


def test_lengths_out_of_range_count_as_the_bounds():
    c = Cache(2, 2, 2, 64, 16, 4, "bf16", [64, 64], seed=8)
    q = c.new(2, 2)
    c.set_lengths([-3, 1000])
    out = sb.cache_decode(c.desc, q, c.lengths, c.table, c.k, c.v, workspace=c.ws)
    want = ref.decode(q, c.k, c.v, c.table, [0, 64], 16, 0, 0)
    finite({"o": out}, want, ("o",))


def test_sequences_may_share_pages():
    c = Cache(2, 4, 2, 64, 16, 8, "bf16", [100, 100], seed=10)
    c.table[1, :5] = c.table[0, :5]
    q = c.new(2, 4)
    out = sb.cache_decode(c.desc, q, c.lengths, c.table, c.k, c.v, workspace=c.ws)
    want = ref.decode(q, c.k, c.v, c.table, [100, 100], 16, 0, 0)
    finite({"o": out}, want, ("o",))


def test_captured_decode_follows_lengths_and_tables():
    c = Cache(3, 8, 2, 128, 16, 40, "bf16", [600, 600, 600], seed=12, window=300, sinks=4,
              weights=True)
    q, kn, vn = c.new(3, 8), c.new(3, 2), c.new(3, 2)
    w = torch.zeros(3, 2, 640, device="cuda")
    nw, out = torch.zeros_like(w), torch.empty_like(q)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:   # two graphs of one workspace, replayed one after the other
        with torch.cuda.graph(graph):
            sb.swin_kvcache_decode(c.desc, q, kn, vn, c.lengths, c.table, c.k, c.v, w, nw, out,
                                   None, c.ws)
    for graph, lengths in zip(graphs * 2, ([600, 1, 304], [0, 305, 303], [17, 599, 2], [600, 600, 600])):
        c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        q.copy_(c.new(3, 8))
        nw.fill_(0)
        graph.replay()
        want = ref.decode(q, c.k, c.v, c.table, lengths, 16, 300, 4, w)
        finite({"o": out, "weights": nw}, want, ("o", "weights"))


@pytest.mark.parametrize("dtype,K,hd,ps", [("bf16", 2, 64, 16), ("f32", 3, 40, 5), ("bf16", 1, 8, 1)])
def test_append_writes_the_last_positions_and_nothing_else(dtype, K, hd, ps):
    B, T, mp = 4, 23, 60 // ps + 1
    lengths, counts = [23, 50, 7, 0], [23, 9, 5, 0]
    c = Cache(B, K, K, hd, ps, mp, dtype, [0] * B, seed=14, kv_stride=2 * K * hd)
    c.set_lengths(lengths)
    x = c.new(B, T, 2 * K)
    k, v = x[:, :, :K], x[:, :, K:]
    want_k, want_v = c.k.clone(), c.v.clone()
    for b, (n, t) in enumerate(zip(lengths, counts)):
        for i in range(t):
            page, row = ref.row_of(c.table, b, n - t + i, ps)
            want_k[page, :, row], want_v[page, :, row] = k[b, i], v[b, i]
    sb.cache_append(c.desc, k, v, c.lengths, c.table, c.k, c.v,
                    counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), workspace=c.ws)
    assert c.status() == 0 and same(c.k, want_k) and same(c.v, want_v)


def test_append_reports_what_it_cannot_write():
    c = Cache(2, 2, 2, 64, 16, 4, "bf16", [0, 0], seed=16)
    k = c.new(2, 10, 2)
    c.set_lengths([10, 4])                       # 10 tokens do not fit a length of 4
    before = c.k.clone()
    sb.cache_append(c.desc, k, k, c.lengths, c.table, c.k, c.v, workspace=c.ws)
    assert c.status() == -1
    for b, n in ((0, 10), (1, 4)):
        for p in range(n):
            page, row = ref.row_of(c.table, b, p, 16)
            before[page, :, row] = k[b, p + 10 - n]
    assert same(c.k, before)
    c.table[1, 0] = c.desc.num_pages
    c.set_lengths([3, 3])
    sb.cache_append(c.desc, k[:, :3].contiguous(), k[:, :3].contiguous(), c.lengths, c.table, c.k,
                    c.v, workspace=c.ws)
    assert c.status() == -1


# K, hd, page, max_pages, lengths, sinks, recent, budget
EVICT = [
    (2, 64, 16, 8, [128, 40, 41, 0, 1], 4, 8, 40),
    (1, 128, 12, 100, [1200, 700], 0, 0, 333),
    (3, 40, 1, 300, [300, 17], 5, 12, 17),            # nothing of the middle stays
    (2, 64, 64, 40, [2500, 2560], 4, 100, 2000),
    (1, 8, 16, 7, [100], 1, 0, 1),
    (1, 64, 16, 4000, [60000], 4, 64, 5000),          # more weights than shared memory holds
    # four blocks to a sequence; rows of weights that start on no 16 bytes; many key
    # heads; four blocks that are full; more positions than registers hold
    (2, 8, 16, 600, [9600, 9001, 4097, 333, 0], 4, 100, 700),
    (2, 16, 3, 3001, [9003, 8192, 4096], 3, 7, 300),
    (8, 8, 16, 300, [4800, 4100, 1025, 1, 4799, 3000, 2049, 0, 500, 4400], 3, 10, 300),
    (1, 8, 64, 2048, [131072], 4, 64, 5000),
    (1, 8, 7, 19201, [134407], 4, 64, 700),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_evict_against_the_reference(case, kind, dtype):
    K, hd, ps, mp, lengths, sinks, recent, budget = case
    B = len(lengths)
    c = Cache(B, K, K, hd, ps, mp, dtype, lengths, seed=18, tables=2, sinks=sinks, recent=recent,
              budget=budget)
    w = torch.rand(B, K, mp * ps, generator=c.gen, device="cuda")
    if kind == "ties":
        w = (w * 3).floor()
    elif kind == "odd":   # NaN, infinities, both zeros, negative numbers
        pick = torch.randint(0, 7, w.shape, generator=c.gen, device="cuda")
        for x, y in enumerate((NAN, float("inf"), float("-inf"), 0.0, -0.0, -1.5)):
            w[pick == x] = y
    kept = torch.full((B, K, budget), -9, dtype=torch.int32, device="cuda")
    nw = torch.full_like(w, 5.0)
    k0, v0 = c.k.clone(), c.v.clone()
    want_k, want_v, host = k0.clone(), v0.clone(), w.cpu().tolist()
    w_before, n_before = w.clone(), c.lengths.clone()
    _, nl = sb.cache_evict(c.desc, w, c.lengths, c.table, c.dst, c.k, c.v, new_weights=nw,
                           kept=kept, workspace=c.ws)
    assert c.status() == 0
    assert same(w, w_before) and torch.equal(c.lengths, n_before)
    assert nl.tolist() == [min(n, budget) for n in lengths]
    at = torch.arange(mp * ps, device="cuda")
    for b, n in enumerate(lengths):
        m = min(n, budget)
        for h in range(K):
            keep = ref.evict(host[b][h], n, sinks, recent, budget)
            assert kept[b, h].tolist() == keep + [-1] * (budget - m)
            pos = torch.tensor(keep, dtype=torch.long, device="cuda")
            want_w = torch.zeros_like(nw[b, h])
            want_w[:m] = w[b, h, pos]
            assert same(nw[b, h], want_w)
            src, dst = c.table[b].long()[pos // ps], c.dst[b].long()[at[:m] // ps]
            want_k[dst, h, at[:m] % ps] = k0[src, h, pos % ps]
            want_v[dst, h, at[:m] % ps] = v0[src, h, pos % ps]
    assert same(c.k, want_k) and same(c.v, want_v)
    # without the list of kept positions
    c.k.copy_(k0)
    c.v.copy_(v0)
    nw2, _ = sb.cache_evict(c.desc, w, c.lengths, c.table, c.dst, c.k, c.v, workspace=c.ws)
    assert same(c.k, want_k) and same(nw2, nw)


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("f32", 64), ("bf16", 128)])
def test_prompt_steps_eviction_steps(dtype, hd):
    """As they are used together: a prompt's attention, its keys and values into
    the cache, steps that accumulate weights, an eviction, and further steps on
    the smaller cache; every step is the reference's on what the cache holds,
    and before the eviction it is the row of the attention over the whole
    sequence."""
    B, H, K, ps, mp, prompt, steps = 2, 4, 2, 16, 12, 100, 9
    c = Cache(B, H, K, hd, ps, mp, dtype, [0] * B, seed=20, tables=2, sinks=2, recent=10, budget=48,
              window=0, weights=True)
    total = prompt + steps
    q, k, v = c.new(B, total, H), c.new(B, total, K), c.new(B, total, K)
    d = sb.make_seq_desc(B, total, H, hd, 0, dtype, kv_heads=K)
    whole, lse = sb.seq_forward(d, q, k, v, want_lse=True)
    want = ref.attention(q, k, v, 0, 0)
    ref.check({"o": whole, "lse": lse}, want, ("o", "lse"))
    c.set_lengths([prompt] * B)
    sb.cache_append(c.desc, k[:, :prompt].contiguous(), v[:, :prompt].contiguous(), c.lengths,
                    c.table, c.k, c.v, workspace=c.ws)
    w = torch.zeros(B, K, mp * ps, device="cuda")
    for t in range(prompt, total):
        c.lengths += 1
        out = sb.cache_decode(c.desc, q[:, t].contiguous(), c.lengths, c.table, c.k, c.v,
                              k_new=k[:, t].contiguous(), v_new=v[:, t].contiguous(), weights=w,
                              workspace=c.ws)
        ref.check({"o": out}, {"o": (want["o"][0][:, t], want["o"][1][:, t])}, ("o",))
    # each step adds one unit of weight per query head
    assert torch.allclose(w.sum(2), torch.full((B, K), steps * H / K, device="cuda"), rtol=1e-4)
    nw, nl = sb.cache_evict(c.desc, w, c.lengths, c.table, c.dst, c.k, c.v, workspace=c.ws)
    assert nl.tolist() == [48] * B
    c.lengths, c.table = nl, c.dst
    for _ in range(3):
        c.lengths += 1
        qn, kn, vn = c.new(B, H), c.new(B, K), c.new(B, K)
        before = nw.clone()
        out = sb.cache_decode(c.desc, qn, c.lengths, c.table, c.k, c.v, k_new=kn, v_new=vn,
                              weights=nw, workspace=c.ws)
        ref_now = ref.decode(qn, c.k, c.v, c.table, c.lengths.tolist(), ps, 0, 0, before)
        finite({"o": out, "weights": nw}, ref_now, ("o", "weights"))
    assert c.status() == 0


def test_wrappers_refuse_what_the_description_does_not_say():
    c = Cache(2, 4, 2, 64, 16, 4, "bf16", [10, 20], seed=22)
    q = c.new(2, 4)
    with pytest.raises(ValueError, match="shape"):
        sb.cache_decode(c.desc, q, c.lengths[:1], c.table, c.k, c.v, workspace=c.ws)
    with pytest.raises(ValueError, match="int32"):
        sb.cache_decode(c.desc, q, c.lengths.long(), c.table, c.k, c.v, workspace=c.ws)
    with pytest.raises(ValueError, match="shape"):
        sb.cache_decode(c.desc, q, c.lengths, c.table, c.k[:5], c.v, workspace=c.ws)
    with pytest.raises(sb.SwinWattnError):   # weights that the workspace has no room for
        sb.cache_decode(c.desc, q, c.lengths, c.table, c.k, c.v,
                        weights=torch.zeros(2, 2, 64, device="cuda"), workspace=c.ws)

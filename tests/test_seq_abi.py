"""Checks of the sequence-attention and cache entry points that need no GPU: the
reference they are tested against, descriptions, pointers, workspaces."""
import ctypes

import pytest
import torch

import seq_reference as ref
from shifted_window_attention_pad_b200 import binding as sb

P = ctypes.c_void_p
GOOD, ODD = P(1 << 20), P((1 << 20) + 2)
AT = lambda n: P((1 << 20) + (n << 28))
BIG = ctypes.c_size_t(1 << 40)


@pytest.fixture(scope="module")
def L():
    from shifted_window_attention_pad_b200 import build
    build.build()
    return sb.lib()


@pytest.mark.parametrize("S,window,sinks,n", [(7, 0, 0, 7), (9, 3, 0, 9), (9, 3, 2, 6), (5, 1, 1, 5)])
def test_reference_gradients_are_those_of_the_forward(S, window, sinks, n):
    """The formulas against autograd of a direct forward and against central
    differences."""
    gen = torch.Generator().manual_seed(S)
    B, H, K, hd = 2, 4, 2, 8
    q, k, v, g = (torch.randn(B, S, h, hd, dtype=torch.float64, generator=gen)
                  for h in (H, K, K, H))
    ref.U[torch.float64] = 0.0
    lengths = [n, max(1, n - 2)]

    def loss(q, k, v):
        total = 0
        for b in range(B):
            m = ref.visible(S, lengths[b], window, sinks, "cpu")[:lengths[b]]
            for h in range(H):
                a = (q[b, :lengths[b], h] @ k[b, :, h // 2].T / hd ** 0.5)
                a = a.masked_fill(~m, float("-inf"))
                total = total + (torch.softmax(a, 1) @ v[b, :, h // 2] * g[b, :lengths[b], h]).sum()
        return total

    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    auto = torch.autograd.grad(loss(*leaves), leaves)
    want = ref.attention(q, k, v, window, sinks, lengths, g)
    for name, a in zip(("dq", "dk", "dv"), auto):
        assert torch.allclose(want[name][0], a, atol=1e-12)
    for x, name in ((0, "dq"), (1, "dk"), (2, "dv")):
        e = torch.zeros_like((q, k, v)[x])
        e.view(-1)[::7] = torch.randn(e.view(-1)[::7].shape, dtype=torch.float64, generator=gen)
        step = [[t + s * e if y == x else t for y, t in enumerate((q, k, v))] for s in (1e-5, -1e-5)]
        slope = (loss(*step[0]) - loss(*step[1])) / 2e-5
        assert abs(float(slope - (want[name][0] * e).sum())) < 1e-7


def _seq(**kw):
    d = sb.make_seq_desc(2, 100, 8, 64, 32, "bf16", kv_heads=2, sinks=4)
    for name, x in kw.items():
        setattr(d, name, x)
    return d


def _cache(**kw):
    d = sb.make_cache_desc(2, 8, 64, 16, 40, 12, "bf16", kv_heads=2, window=32, sinks=4, recent=8,
                           budget=40, weights=True)
    for name, x in kw.items():
        setattr(d, name, x)
    return d


@pytest.mark.parametrize("field,value", [
    ("B", 0), ("S", 0), ("S", (1 << 30) + 1), ("heads", 0), ("heads", 7), ("kv_heads", 0),
    ("kv_heads", 3), ("head_dim", 12), ("head_dim", 0), ("head_dim", 264), ("window", -1),
    ("sinks", -1), ("q_stride", 256), ("q_stride", 513), ("kv_stride", -8), ("kv_stride", 64)])
def test_bad_sequence_descriptions(L, field, value):
    d, n = _seq(**{field: value}), ctypes.c_size_t(0)
    assert L.swin_seqattn_path(ctypes.byref(d)) == -1
    assert L.swin_seqattn_workspace_size(ctypes.byref(d), ctypes.byref(n)) == -1
    assert L.swin_seqattn_fwd(ctypes.byref(d), AT(0), AT(1), AT(2), None, AT(3), None, GOOD, BIG,
                              None) == -1


@pytest.mark.parametrize("field,value", [
    ("B", 0), ("heads", 0), ("heads", 7), ("kv_heads", 3), ("head_dim", 4), ("page_size", 0),
    ("page_size", 65537), ("num_pages", 0), ("max_pages", 0), ("max_pages", 1 << 28),
    ("window", -1), ("sinks", -1), ("budget", -1), ("budget", 12 * 16 + 1), ("recent", -1),
    ("q_stride", 100), ("kv_stride", 129)])
def test_bad_cache_descriptions(L, field, value):
    d, n = _cache(**{field: value}), ctypes.c_size_t(0)
    assert L.swin_kvcache_workspace_size(ctypes.byref(d), ctypes.byref(n)) == -1


def test_bad_dtype(L):
    n = ctypes.c_size_t(0)
    assert L.swin_seqattn_path(ctypes.byref(_seq(dtype=5))) == -2
    assert L.swin_kvcache_workspace_size(ctypes.byref(_cache(dtype=5)), ctypes.byref(n)) == -2
    with pytest.raises(ValueError):
        sb.make_seq_desc(1, 1, 1, 64, 0, "f16")
    assert sb.make_seq_desc(1, 1, 1, 64, 0, "f32").dtype == sb.SWIN_DTYPE_F32


def test_paths(L):
    for hd, dtype, want in ((64, "bf16", 1), (128, "bf16", 1), (80, "bf16", 1), (136, "bf16", 0),
                            (64, "f32", 0)):
        d = sb.make_seq_desc(1, 300, 4, hd, 0, dtype)
        assert sb.swin_seqattn_path(d) == want, (hd, dtype)
        d.flags = sb.SWIN_FLAG_FORCE_GENERIC
        assert sb.swin_seqattn_path(d) == 0


@pytest.mark.parametrize("bad", range(4))
def test_forward_pointers(L, bad):
    d = ctypes.byref(_seq())
    for x in (None, ODD):
        a = [AT(0), AT(1), AT(2), AT(3)]
        a[bad] = x
        assert L.swin_seqattn_fwd(d, *a[:3], None, a[3], None, GOOD, BIG, None) == -1


def test_forward_refuses_overlap_and_workspaces(L):
    d = ctypes.byref(_seq())
    for x in range(3):   # out on q, k or v
        assert L.swin_seqattn_fwd(d, AT(0), AT(1), AT(2), None, AT(x), None, GOOD, BIG, None) == -1
    args = (d, AT(0), AT(1), AT(2), None, AT(3), None)
    assert L.swin_seqattn_fwd(d, AT(0), AT(1), AT(2), P((1 << 20) + 2), AT(3), None, GOOD, BIG,
                              None) == -1
    assert L.swin_seqattn_fwd(*args, None, BIG, None) == -3
    assert L.swin_seqattn_fwd(*args, P((1 << 20) + 16), BIG, None) == -3
    n = sb.swin_seqattn_workspace_size(_seq())
    assert L.swin_seqattn_fwd(*args, GOOD, ctypes.c_size_t(n - 1), None) == -3


@pytest.mark.parametrize("bad", range(9))
def test_backward_pointers(L, bad):
    d = ctypes.byref(_seq())
    for x in (None, ODD):
        a = [AT(y) for y in range(9)]   # q k v out lse dout dq dk dv
        a[bad] = x
        assert L.swin_seqattn_bwd(d, *a[:3], None, *a[3:], GOOD, BIG, None) == -1


def test_backward_refuses_shared_outputs(L):
    d = ctypes.byref(_seq())
    for x, y in ((6, 7), (7, 8), (6, 8), (6, 3), (6, 5), (7, 5), (8, 5), (6, 0), (7, 1), (8, 2)):
        a = [AT(z) for z in range(9)]
        a[x] = a[y]
        assert L.swin_seqattn_bwd(d, *a[:3], None, *a[3:], GOOD, BIG, None) == -1, (x, y)


def test_workspace_grows_with_what_it_holds():
    """Header and (lse, D) of every row; with few key heads, or sinks in front
    of a long sequence, fp32 partials of dk and dv."""
    a256 = lambda x: (x + 255) // 256 * 256
    d = sb.make_seq_desc(8, 4096, 32, 64, 512, "bf16")
    assert sb.swin_seqattn_workspace_size(d) == 256 + 8 * 4096 * 32 * 8
    one = sb.make_seq_desc(1, 256, 4, 64, 0, "bf16", kv_heads=1)
    assert sb.swin_seqattn_workspace_size(one) == 256 + a256(256 * 4 * 8) + 4 * 2 * 256 * 64 * 4
    sinks = sb.make_seq_desc(8, 4096, 32, 64, 512, "bf16", sinks=4)
    # one sink tile of 128 keys for each of 8 x 32 heads, four chunks of 1024 queries
    assert (sb.swin_seqattn_workspace_size(sinks) - sb.swin_seqattn_workspace_size(d)
            == 2 * 8 * 32 * 4 * 128 * 64 * 4)
    # sinks that the window covers are no sinks
    wide = sb.make_seq_desc(8, 4096, 32, 64, 4096, "bf16", sinks=4)
    assert sb.swin_seqattn_workspace_size(wide) == sb.swin_seqattn_workspace_size(d)


def test_cache_calls_refuse_bad_arguments(L):
    d = ctypes.byref(_cache())
    app = [AT(0), AT(1), None, AT(2), AT(3), AT(4), AT(5)]
    assert L.swin_kvcache_append(d, 0, *app, GOOD, BIG, None) == -1
    for x in (0, 1, 3, 4, 5, 6):
        bad = list(app)
        bad[x] = None
        assert L.swin_kvcache_append(d, 1, *bad, GOOD, BIG, None) == -1, x
    assert L.swin_kvcache_append(d, 1, *app[:5], AT(4), AT(4), GOOD, BIG, None) == -1
    assert L.swin_kvcache_append(d, 1, *app, None, BIG, None) == -3
    # q k_new v_new lengths table kc vc weights new_weights out lse
    dec = [AT(0), AT(1), AT(2), AT(3), AT(4), AT(5), AT(6), AT(7), AT(7), AT(8), None]
    for x in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9):
        bad = list(dec)
        bad[x] = None   # k_new without v_new, weights without new_weights
        assert L.swin_kvcache_decode(d, *bad, GOOD, BIG, None) == -1, x
    assert L.swin_kvcache_decode(ctypes.byref(_cache(flags=0)), *dec, GOOD, BIG, None) == -1
    n = sb.swin_kvcache_workspace_size(_cache())
    assert L.swin_kvcache_decode(d, *dec, GOOD, ctypes.c_size_t(n - 1), None) == -3
    # weights lengths table dst kc vc new_weights new_lengths kept
    ev = [AT(0), AT(1), AT(2), AT(3), AT(4), AT(5), AT(6), AT(7), None]
    for x in range(8):
        bad = list(ev)
        bad[x] = None
        assert L.swin_kvcache_evict(d, *bad, GOOD, BIG, None) == -1, x
    for x, y in ((6, 0), (7, 1), (3, 2), (5, 4)):   # in place
        bad = list(ev)
        bad[x] = bad[y]
        assert L.swin_kvcache_evict(d, *bad, GOOD, BIG, None) == -1, (x, y)
    for kw in (dict(budget=0), dict(budget=11), dict(recent=37)):
        assert L.swin_kvcache_evict(ctypes.byref(_cache(**kw)), *ev, GOOD, BIG, None) == -1, kw
    assert L.swin_kvcache_evict(d, *ev, P((1 << 20) + 128), BIG, None) == -3


def test_outputs_that_overlap_inputs_are_refused(L):
    d, c = ctypes.byref(_seq()), ctypes.byref(_cache())
    behind = lambda n: P((1 << 20) + (n << 28) + 256)   # inside what AT(n) holds
    # q k v out lse: lse on each of the others
    for x in range(4):
        assert L.swin_seqattn_fwd(d, AT(0), AT(1), AT(2), None, AT(3), behind(x), GOOD, BIG,
                                  None) == -1, x
    # q k v out lse dout dq dk dv: a gradient inside out, lse or dout
    for x in (6, 7, 8):
        for y in (3, 4, 5):
            a = [AT(z) for z in range(9)]
            a[x] = behind(y)
            assert L.swin_seqattn_bwd(d, *a[:3], None, *a[3:], GOOD, BIG, None) == -1, (x, y)
    # k v counts lengths table kc vc: one cache inside the other, tokens inside a cache
    for x, y in ((6, 5), (0, 5), (0, 6), (1, 5), (1, 6)):
        a = [AT(0), AT(1), None] + [AT(z) for z in range(3, 7)]
        a[x] = behind(y)
        assert L.swin_kvcache_append(c, 1, *a, GOOD, BIG, None) == -1, (x, y)
    # q k_new v_new lengths table kc vc weights new_weights out lse
    for x, y in ((6, 5), (9, 0), (9, 1), (9, 2), (9, 5), (9, 6), (10, 9), (8, 7)):
        a = [AT(z) for z in range(11)]
        a[x] = behind(y)
        assert L.swin_kvcache_decode(c, *a, GOOD, BIG, None) == -1, (x, y)
    # weights lengths table dst kc vc new_weights new_lengths kept
    a = [AT(z) for z in range(8)] + [None]
    a[5] = behind(4)
    assert L.swin_kvcache_evict(c, *a, GOOD, BIG, None) == -1


def test_caches_past_what_is_addressed_are_refused():
    """Positions are counted in 32 bits, with room for a tile behind the last."""
    long = dict(page_size=65536, max_pages=1 << 14, num_pages=1 << 15)
    assert sb.swin_kvcache_workspace_size(_cache(**long)) > 0
    with pytest.raises(sb.SwinWattnError):
        sb.swin_kvcache_workspace_size(_cache(**dict(long, max_pages=(1 << 14) + 1)))
    with pytest.raises(sb.SwinWattnError):
        sb.swin_kvcache_workspace_size(_cache(num_pages=0x7fffffff, page_size=65536, max_pages=1,
                                              head_dim=256))


def test_wrappers_refuse_host_tensors():
    d = sb.make_seq_desc(1, 4, 2, 64, 0, "bf16")
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sb.seq_forward(d, x, x, x)


def test_description_of_parts_of_a_projection():
    qkv = torch.zeros(2, 5, 12, 64)
    d = sb.seq_desc_for(qkv[:, :, :8], qkv[:, :, 8:10], window=0)
    assert (d.B, d.S, d.heads, d.kv_heads, d.head_dim) == (2, 5, 8, 2, 64)
    assert d.q_stride == d.kv_stride == 768
    one = sb.seq_desc_for(qkv[:1, :1, :8], qkv[:1, :1, 8:10], window=0)
    assert one.q_stride == one.kv_stride == 0      # a single token has no stride
    whole = torch.zeros(2, 5, 8, 64)
    assert sb.seq_desc_for(whole, whole, window=0).q_stride == 0

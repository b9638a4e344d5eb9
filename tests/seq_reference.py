"""Plain 64-bit implementations of sequence attention and of the paged cache's
operations, with the bounds their results are held to.

Bounds. A rounding to a type is off by at most u = finfo.eps / 2 of the value
(bf16 2^-8, fp32 2^-24). The kernels form logits, softmax statistics and sums in
fp32 and round to bf16 (where the inputs are bf16): P before P V, dS before
dS K and dS^T Q, P before P^T dO, and the outputs. So, element by element,
  |o - ref|  <= u |ref| + (u + s) sum_j P |v|
  |dv - ref| <= u |ref| + (u + s) sum_i P |dO|
  |dq - ref| <= u |ref| + scale sum_j ((u + s) |dS| + P dD_i) |k|
(dk as dq), dD_i = (2 u + s) sum_d |dO| |o| from D = dO.o of the rounded out, and
s = 2^-24 (4 n + 8 hd A): fp32 sums over n keys, and logits of hd products whose
magnitudes add to at most A = scale |q| |k| (an error of a logit is a relative
error of P). The weights' and lse's own bounds follow in the same way."""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def visible(S, n, window, sinks, device):
    i = torch.arange(S, device=device)[:, None]
    j = torch.arange(S, device=device)[None, :]
    m = (j <= i) & (i < n)
    if window:
        m &= (i - j < window) | (j < sinks)
    return m


def attention(q, k, v, window, sinks, lengths=None, dout=None):
    """{name: (value, bound)} for o, lse (and dq, dk, dv), in float64."""
    B, S, H, hd = q.shape
    K, u, dev = k.shape[2], U[q.dtype], q.device
    f = lambda t: t.detach().double()
    # what padding holds is not used
    n_of = [S if lengths is None else min(max(int(lengths[b]), 0), S) for b in range(B)]
    real = torch.zeros(B, S, 1, 1, dtype=torch.bool, device=dev)
    for b, n in enumerate(n_of):
        real[b, :n] = True
    q, k, v = (torch.where(real, f(t), 0.0) for t in (q, k, v))
    out, lse = torch.zeros_like(q), torch.zeros(B, S, H, dtype=torch.float64, device=dev)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    res = {}
    if dout is not None:
        g = torch.where(real, f(dout), 0.0)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        bq, bk, bv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    scale = hd ** -0.5
    for b, n in enumerate(n_of):
        if n == 0:
            continue
        m = visible(n, n, window, sinks, dev)
        for h in range(H):
            c = h // (H // K)
            qh, kh, vh = q[b, :n, h], k[b, :n, c], v[b, :n, c]
            a = (qh @ kh.T * scale).masked_fill(~m, float("-inf"))
            L = torch.logsumexp(a, 1)
            p = torch.exp(a - L[:, None])
            A = float(scale * qh.norm(dim=1).max() * kh.norm(dim=1).max())
            s = 2.0 ** -24 * (4 * n + 8 * hd * A)
            o = p @ vh
            out[b, :n, h], lse[b, :n, h] = o, L
            bo[b, :n, h] = u * o.abs() + (u + s) * (p @ vh.abs())
            bl[b, :n, h] = s + 2.0 ** -22 * L.abs()
            if dout is not None:
                gh = g[b, :n, h]
                ds = p * (gh @ vh.T - (gh * o).sum(1, keepdim=True))
                dD = (2 * u + s) * (gh.abs() * o.abs()).sum(1, keepdim=True) + \
                    u * (gh.abs() * (p @ vh.abs())).sum(1, keepdim=True)
                sg = s * p * (gh.norm(dim=1).max() * vh.norm(dim=1).max())
                e = scale * ((u + s) * ds.abs() + p * dD + sg)
                dq[b, :n, h] = ds @ kh * scale
                bq[b, :n, h] = e @ kh.abs()
                dk[b, :n, c] += ds.T @ qh * scale
                bk[b, :n, c] += e.T @ qh.abs()
                dv[b, :n, c] += p.T @ gh
                bv[b, :n, c] += (u + s) * (p.T @ gh.abs())
    res["o"], res["lse"] = (out, bo), (lse, bl)
    if dout is not None:
        res["dq"] = (dq, bq + u * dq.abs())
        res["dk"] = (dk, bk + u * dk.abs())
        res["dv"] = (dv, bv + u * dv.abs())
    return res


def check(got, want, names):
    for name in names:
        ref, bound = want[name]
        x = got[name].double()
        assert x.shape == ref.shape, name
        assert torch.isfinite(x).all(), name
        over = (x - ref).abs() - bound - 1e-30
        worst = float(over.max())
        assert worst <= 0, (name, worst, float(((x - ref).abs() / (bound + 1e-30)).max()))


# ---- paged cache -------------------------------------------------------------------
def row_of(table, b, pos, page_size):
    return int(table[b, pos // page_size]), pos % page_size


def gather(cache, table, b, head, positions, page_size):
    rows = [row_of(table, b, p, page_size) for p in positions]
    if not rows:
        return cache.new_zeros((0, cache.shape[-1]))
    pages, at = zip(*rows)
    return cache[list(pages), head, list(at)]


def decode(q, k_cache, v_cache, table, lengths, page_size, window, sinks, weights=None):
    """{name: (value, bound)} of o, lse (and weights) for caches that hold the
    new token already."""
    B, H, hd = q.shape
    K, u, dev = k_cache.shape[1], U[q.dtype], q.device
    o = torch.zeros(B, H, hd, dtype=torch.float64, device=dev)
    lse = torch.full((B, H), float("-inf"), dtype=torch.float64, device=dev)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    w = bw = None
    if weights is not None:
        w = weights.double().clone()
        bw = torch.zeros_like(w)
    table = table.cpu()
    scale = hd ** -0.5
    for b in range(B):
        n = int(lengths[b])
        see = [p for p in range(n) if not window or p >= n - window or p < sinks]
        if not see:
            continue
        for c in range(K):
            kk = gather(k_cache, table, b, c, see, page_size).double()
            vv = gather(v_cache, table, b, c, see, page_size).double()
            hs = slice(c * (H // K), (c + 1) * (H // K))
            qq = q[b, hs].double()
            a = qq @ kk.T * scale
            L = torch.logsumexp(a, 1)
            p = torch.exp(a - L[:, None])
            A = float(scale * qq.norm(dim=1).max() * kk.norm(dim=1).max())
            s = 2.0 ** -24 * (4 * len(see) + 8 * hd * A)
            o[b, hs], lse[b, hs] = p @ vv, L
            bo[b, hs] = u * (p @ vv).abs() + (u + s) * (p @ vv.abs())
            bl[b, hs] = s + 2.0 ** -22 * L.abs()
            if w is not None:
                at = torch.tensor(see, device=dev)
                w[b, c, at] += p.sum(0)
                bw[b, c, at] = s * p.sum(0) + 2.0 ** -23 * w[b, c, at].abs()
    res = {"o": (o, bo), "lse": (lse, bl)}
    if w is not None:
        res["weights"] = (w, bw)
    return res


def evict(weights, n, sinks, recent, budget):
    """Kept positions of one kv head (a list of Python numbers as weights)."""
    if n <= budget:
        return list(range(n))
    rank = lambda p: (0, 0.0) if weights[p] != weights[p] else (-1, -weights[p])
    middle = sorted(range(sinks, n - recent), key=lambda p: (*rank(p), p))
    return sorted([*range(sinks), *middle[:budget - sinks - recent], *range(n - recent, n)])

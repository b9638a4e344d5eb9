"""Sequence attention (sliding window with sink tokens), single-token attention
over a paged key-value cache, filling that cache, and eviction from it by
accumulated attention weight: what each computes in elementary torch
operations, the framework's own calls, and the cases they are measured on.

Conventions. q [B, S, heads, hd], k and v [B, S, kv_heads, hd]; query head h
reads kv head h // (heads // kv_heads). Key j is visible to query i of a
sequence of `length` tokens when j <= i < length and (window == 0, or
i - j < window, or j < sinks). Tokens at and beyond a sequence's length get
zeros. A cache is [pages, kv_heads, page_size, hd]; position p of sequence b
is row p % page_size of page page_table[b, p // page_size].
"""
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------------
def _seq(op, B, S, heads, kv_heads, hd, window, sinks, dtype, ragged=False, fused=False,
         len_seed=0, **kw):
    return dict(op=op, B=B, S=S, heads=heads, kv_heads=kv_heads, hd=hd, window=window,
                sinks=sinks, dtype=dtype, ragged=ragged, fused=fused, len_seed=len_seed, **kw)


def _cache(op, B, min_len, max_len, heads, kv_heads, hd, page, dtype, len_seed=0, **kw):
    return dict(op=op, B=B, min_len=min_len, max_len=max_len, heads=heads, kv_heads=kv_heads,
                hd=hd, page=page, dtype=dtype, len_seed=len_seed, **kw)


def listed():
    return [
        # a short ragged history of a small model (the 4 heads x 32 of the ragged workload)
        _seq("fwd", 2, 90, 4, 4, 32, 32, 1, "bf16", ragged=True, name="seq-fwd-short"),
        # a long prompt with a wide window, four query heads to a key head
        _seq("fwd", 1, 16384, 16, 4, 128, 4096, 4, "bf16", name="seq-fwd-long"),
        # fp32 training of a small model on one grid row of 544 tokens
        _seq("train", 1, 544, 8, 8, 64, 128, 2, "f32", name="seq-train-f32"),
        # a training step on ragged sequences, q, k, v cut from one fused projection
        _seq("train", 2, 4096, 16, 16, 64, 512, 4, "bf16", ragged=True, fused=True,
             name="seq-train-window"),
        # a training step with no window at all (plain causal), shared key heads
        _seq("train", 1, 8192, 8, 2, 128, 0, 0, "bf16", name="seq-train-causal"),
        # the smallest serving step: few short fp32 sequences, odd page size, a window
        _cache("decode", 4, 1, 700, 8, 8, 64, 12, "f32", window=256, sinks=4, weights=False,
               name="decode-small"),
        # a serving batch with lengths from short to long
        _cache("decode", 64, 200, 8192, 16, 4, 128, 16, "bf16", window=0, sinks=0, weights=False,
               name="decode-batch"),
        # two long sequences whose attention weights are accumulated for eviction
        _cache("decode", 2, 40000, 65536, 16, 2, 128, 64, "bf16", window=0, sinks=0, weights=True,
               name="decode-long-weights"),
        # one new token of every sequence goes into the cache
        _cache("append", 64, 1, 4096, 4, 4, 128, 16, "bf16", tokens=1, name="append-token"),
        # prompts go into the cache
        _cache("append", 8, 300, 4096, 8, 8, 128, 16, "bf16", tokens=4096, name="append-prompt"),
        # a small cache is cut to a quarter
        _cache("evict", 4, 200, 1024, 4, 4, 64, 16, "f32", sinks=4, recent=32, budget=256,
               name="evict-small"),
        # long caches are cut to 4096 positions
        _cache("evict", 8, 9000, 32768, 8, 8, 128, 16, "bf16", sinks=4, recent=512, budget=4096,
               name="evict-long"),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


_MOST = 5.0e11      # FLOPs of the costliest listed sequence case
_MOST_F32 = 2.0e10  # the same for fp32, which has no matrix instructions


def draw(rng):
    op = rng.choice(["fwd", "train", "train", "decode", "decode", "append", "evict"])
    hd = rng.choice([32, 64, 64, 128, 128, 80])
    group = rng.choice([1, 1, 2, 4, 8])
    kv_heads = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    len_seed = rng.randrange(1 << 20)
    if op in ("fwd", "train"):
        while True:
            S = _log_int(rng, 16, 16384)
            window = rng.choice([0, _log_int(rng, 16, 8192), _log_int(rng, 16, 8192)])
            case = _seq(op, rng.choice([1, 1, 2, 3, 5]), S, kv_heads * group, kv_heads, hd, window,
                        rng.choice([0, 1, 4, 19]), dtype, rng.random() < 0.5, rng.random() < 0.4,
                        len_seed)
            # head_dim 80 runs without matrix instructions in both types
            most = _MOST_F32 if dtype == "f32" or hd == 80 else _MOST
            if work(case)["flops"] <= most:
                return case
    while True:
        B = _log_int(rng, 1, 96)
        max_len = _log_int(rng, 16, 65536)
        case = _cache(op, B, rng.choice([1, max(1, max_len // 3), max_len]), max_len,
                      kv_heads * group, kv_heads, hd, rng.choice([16, 16, 32, 64, 12, 128]), dtype,
                      len_seed)
        if op == "decode":
            case.update(window=rng.choice([0, 0, _log_int(rng, 16, 8192)]),
                        sinks=rng.choice([0, 4, 7]), weights=rng.random() < 0.4)
        elif op == "append":
            case.update(tokens=rng.choice([1, 3, _log_int(rng, 1, max_len)]))
        else:
            budget = _log_int(rng, 8, max(9, max_len))
            sinks = rng.choice([0, 2, 4])
            case.update(budget=budget, sinks=sinks, recent=rng.randrange(0, budget - sinks + 1))
        elem = 2 if dtype == "bf16" else 4
        if B * max_len * kv_heads * hd * 2 * elem <= 1_200_000_000:
            return case


def _lengths(case):
    rng = random.Random(case["len_seed"])
    if "S" in case:
        S = case["S"]
        return [rng.randint(max(1, S // 3), S) if case["ragged"] else S for _ in range(case["B"])]
    return [rng.randint(case["min_len"], case["max_len"]) for _ in range(case["B"])]


def _counts(case, lengths):
    """Tokens that an append brings to each sequence."""
    return [min(n, case["tokens"]) for n in lengths]


def _visible(n, window, sinks):
    """Positions a query at position n - 1 sees."""
    return n if window == 0 else min(n, window + sinks)


def work(case):
    lengths, elem = _lengths(case), 2 if case["dtype"] == "bf16" else 4
    hd, H, K, tot = case["hd"], case["heads"], case["kv_heads"], sum(lengths)
    if case["op"] in ("fwd", "train"):
        window, sinks = case["window"], case["sinks"]
        pairs = 0
        for n in lengths:
            m = n if window == 0 else min(n, window + sinks)   # rows that see all before them
            pairs += m * (m + 1) // 2 + (n - m) * (window + sinks)
        q, kv = tot * H * hd * elem, tot * K * hd * elem
        if case["op"] == "fwd":
            return {"bytes": 2 * q + 2 * kv + tot * H * 4, "flops": 4 * hd * H * pairs}
        return {"bytes": 4 * q + 4 * kv + tot * H * 4, "flops": 14 * hd * H * pairs}
    row = K * hd * elem
    if case["op"] == "decode":
        seen = sum(_visible(n, case["window"], case["sinks"]) for n in lengths)
        b = 2 * seen * row + case["B"] * (2 * H * hd * elem + H * 4 + 2 * row)
        if case["weights"]:
            b += 8 * tot * K
        return {"bytes": b, "flops": 4 * hd * H * seen}
    if case["op"] == "append":
        return {"bytes": 4 * sum(_counts(case, lengths)) * row, "flops": 0}
    kept = sum(min(n, case["budget"]) for n in lengths)
    return {"bytes": 4 * kept * row + 4 * tot * K + 8 * kept * K, "flops": 0}


# ---- inputs ------------------------------------------------------------------------
def _page_tables(case, lengths, tables, gen):
    """`tables` page tables over one pool, pages in shuffled order; unused
    entries are -1. Returns them and the number of pages in the pool."""
    ps, out, need = case["page"], [], 0
    width = -(-case["max_len"] // ps)
    for lens in tables:
        need += sum(-(-n // ps) for n in lens)
    ids = torch.randperm(need, generator=gen).tolist()
    at = 0
    for lens in tables:
        t = torch.full((case["B"], width), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            m = -(-n // ps)
            t[b, :m] = torch.tensor(ids[at:at + m], dtype=torch.int32)
            at += m
        out.append(t.cuda())
    return out, need


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    dt, lengths = DTYPES[case["dtype"]], _lengths(case)
    B, H, K, hd = case["B"], case["heads"], case["kv_heads"], case["hd"]
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda").to(dt)
    st = {"case": case}
    if case["op"] in ("fwd", "train"):
        S = case["S"]
        if case["fused"]:
            qkv = normal(B, S, H + 2 * K, hd)
            st["q"], st["k"], st["v"] = qkv[:, :, :H], qkv[:, :, H:H + K], qkv[:, :, H + K:]
        else:
            st["q"], st["k"], st["v"] = normal(B, S, H, hd), normal(B, S, K, hd), normal(B, S, K, hd)
        st["lengths"] = (torch.tensor(lengths, dtype=torch.int32).cuda() if case["ragged"] else None)
        if case["op"] == "train":
            st["dout"] = normal(B, S, H, hd)
        if own:
            from shifted_window_attention_pad_b200 import binding as sb
            st["desc"] = sb.seq_desc_for(st["q"], st["k"], window=case["window"], sinks=case["sinks"])
            st["ws"] = sb.new_seq_workspace(st["desc"])
        return st
    ps = case["page"]
    st["lengths"] = torch.tensor(lengths, dtype=torch.int32).cuda()
    tables = [lengths]
    if case["op"] == "evict":
        tables.append([min(n, case["budget"]) for n in lengths])
    tabs, pages = _page_tables(case, lengths, tables, cpu)
    width = tabs[0].shape[1]
    st["page_table"] = tabs[0]
    st["k_cache"], st["v_cache"] = normal(pages, K, ps, hd), normal(pages, K, ps, hd)
    # weights that earlier steps left: most positions little, a few much
    if case["op"] == "evict" or case.get("weights"):
        u = torch.rand(B, K, width * ps, generator=gen, device="cuda")
        st["weights"] = u ** 8 * 16
    if case["op"] == "decode":
        st["q"], st["k_new"], st["v_new"] = normal(B, H, hd), normal(B, K, hd), normal(B, K, hd)
        if case["weights"]:
            st["new_weights"] = torch.zeros_like(st["weights"])
    elif case["op"] == "append":
        T = min(case["tokens"], case["max_len"])
        kv = normal(B, T, 2 * K, hd)   # keys and values cut from one projection
        st["k"], st["v"] = kv[:, :, :K], kv[:, :, K:]
        st["counts"] = torch.tensor(_counts(case, lengths), dtype=torch.int32).cuda()
    else:
        st["dst_page_table"] = tabs[1]
        st["new_weights"] = torch.empty_like(st["weights"])
        st["new_lengths"] = torch.empty_like(st["lengths"])
        st["kept"] = torch.empty(B, K, case["budget"], dtype=torch.int32, device="cuda")
    if own:
        from shifted_window_attention_pad_b200 import binding as sb
        more = {k: case[k] for k in ("window", "sinks", "recent", "budget", "weights") if k in case}
        kv_stride = 2 * K * hd if case["op"] == "append" else 0
        st["desc"] = sb.make_cache_desc(B, H, hd, ps, pages, width, case["dtype"], kv_heads=K,
                                        kv_stride=kv_stride, **more)
        st["ws"] = sb.new_cache_workspace(st["desc"])
    return st


# ---- one pass ----------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    from shifted_window_attention_pad_b200 import binding as sb
    op = st["case"]["op"]
    if op in ("fwd", "train"):
        d, q, k, v, n, ws = st["desc"], st["q"], st["k"], st["v"], st["lengths"], st["ws"]
        out, lse = sb.seq_forward(d, q, k, v, lengths=n, want_lse=True, workspace=ws)
        if op == "fwd":
            return [out, lse]
        dq, dk, dv = sb.seq_backward(d, q, k, v, out, lse, st["dout"], lengths=n, workspace=ws)
        return [out, lse, dq, dk, dv]
    if op == "decode":
        out, lse = sb.cache_decode(st["desc"], st["q"], st["lengths"], st["page_table"],
                                   st["k_cache"], st["v_cache"], k_new=st["k_new"],
                                   v_new=st["v_new"], weights=st.get("weights"),
                                   new_weights=st.get("new_weights"), want_lse=True,
                                   workspace=st["ws"])
        res = [out, lse, st["k_cache"], st["v_cache"]]
        return res + [st["new_weights"]] if st["case"]["weights"] else res
    if op == "append":
        sb.cache_append(st["desc"], st["k"], st["v"], st["lengths"], st["page_table"],
                        st["k_cache"], st["v_cache"], counts=st["counts"], workspace=st["ws"])
        return [st["k_cache"], st["v_cache"]]
    sb.cache_evict(st["desc"], st["weights"], st["lengths"], st["page_table"],
                   st["dst_page_table"], st["k_cache"], st["v_cache"],
                   new_weights=st["new_weights"], new_lengths=st["new_lengths"], kept=st["kept"],
                   workspace=st["ws"])
    return [st["k_cache"], st["v_cache"], st["new_weights"], st["new_lengths"], st["kept"]]


_BLOCK = 512   # queries at a time


def _key_ranges(i0, i1, window, sinks):
    """Keys that queries i0 .. i1 - 1 can see, as one or two ranges."""
    lo = 0 if window == 0 else max(0, i0 - window + 1)
    if lo <= sinks:
        return torch.arange(0, i1, device="cuda")
    return torch.cat([torch.arange(0, sinks, device="cuda"), torch.arange(lo, i1, device="cuda")])


def _plain_seq(st):
    c, dt = st["case"], st["q"].dtype
    B, S, H, K, hd = c["B"], c["S"], c["heads"], c["kv_heads"], c["hd"]
    G, scale = H // K, hd ** -0.5
    train = c["op"] == "train"
    n = st["lengths"]
    if n is None:
        n = torch.full((B,), S, dtype=torch.int32, device="cuda")
    # [B, K, G, S, hd] and [B, K, 1, S, hd]
    q = st["q"].float().reshape(B, S, K, G, hd).permute(0, 2, 3, 1, 4)
    k, v = (st[x].float().permute(0, 2, 1, 3).unsqueeze(2) for x in ("k", "v"))
    out = torch.zeros(B, K, G, S, hd, device="cuda")
    lse = torch.zeros(B, K, G, S, device="cuda")
    if train:
        do = st["dout"].float().reshape(B, S, K, G, hd).permute(0, 2, 3, 1, 4)
        dq, dk, dv = torch.zeros_like(out), torch.zeros_like(k), torch.zeros_like(v)
    for i0 in range(0, S, _BLOCK):
        i1 = min(S, i0 + _BLOCK)
        j = _key_ranges(i0, i1, c["window"], c["sinks"])
        i = torch.arange(i0, i1, device="cuda")[:, None]
        see = j <= i
        if c["window"]:
            see &= (i - j < c["window"]) | (j < c["sinks"])
        real = (i < n[:, None, None])[:, None, None]               # [B, 1, 1, rows, 1]
        kj, vj = k[:, :, :, j], v[:, :, :, j]
        a = torch.matmul(q[:, :, :, i0:i1], kj.transpose(-1, -2)) * scale
        a = a.masked_fill(~see, float("-inf"))
        m = a.amax(-1, keepdim=True)
        p = torch.exp(a - m)
        z = p.sum(-1, keepdim=True)
        p = p / z * real
        o = torch.matmul(p, vj)
        out[:, :, :, i0:i1] = o
        lse[:, :, :, i0:i1] = ((m + torch.log(z)) * real)[..., 0]
        if train:
            g = do[:, :, :, i0:i1] * real
            dp = torch.matmul(g, vj.transpose(-1, -2))
            ds = p * (dp - (g * o).sum(-1, keepdim=True)) * scale
            dq[:, :, :, i0:i1] = torch.matmul(ds, kj)
            dk[:, :, 0].index_add_(2, j, torch.matmul(ds.transpose(-1, -2), q[:, :, :, i0:i1]).sum(2))
            dv[:, :, 0].index_add_(2, j, torch.matmul(p.transpose(-1, -2), g).sum(2))
    back_q = lambda t: t.permute(0, 3, 1, 2, 4).reshape(B, S, H, hd).to(dt)
    back_k = lambda t: t[:, :, 0].permute(0, 2, 1, 3).to(dt)
    res = [back_q(out), lse.permute(0, 3, 1, 2).reshape(B, S, H).contiguous()]
    return res + [back_q(dq), back_k(dk), back_k(dv)] if train else res


def _rows(st, b, n):
    """Page and row of positions 0 .. n - 1 of sequence b."""
    p = torch.arange(n, device="cuda")
    ps = st["case"]["page"]
    return st["page_table"][b].long()[p // ps], p % ps


def _run_plain(st):
    c = st["case"]
    if c["op"] in ("fwd", "train"):
        return _plain_seq(st)
    B, H, K, hd, ps = c["B"], c["heads"], c["kv_heads"], c["hd"], c["page"]
    kc, vc, lengths = st["k_cache"], st["v_cache"], _lengths(c)
    if c["op"] == "append":
        for b, (n, t) in enumerate(zip(lengths, _counts(c, lengths))):
            page, row = (x[n - t:] for x in _rows(st, b, n))
            kc[page, :, row], vc[page, :, row] = st["k"][b, :t], st["v"][b, :t]
        return [kc, vc]
    if c["op"] == "decode":
        out = torch.empty(B, H, hd, dtype=kc.dtype, device="cuda")
        lse = torch.empty(B, H, device="cuda")
        for b, n in enumerate(lengths):
            page, row = _rows(st, b, n)
            kc[page[-1], :, row[-1]], vc[page[-1], :, row[-1]] = st["k_new"][b], st["v_new"][b]
            j = _key_ranges(n - 1, n, c["window"], c["sinks"])
            k, v = (x[page[j], :, row[j]].float().transpose(0, 1) for x in (kc, vc))  # [K, n, hd]
            a = torch.matmul(st["q"][b].float().reshape(K, H // K, hd), k.transpose(1, 2)) * hd ** -0.5
            m = a.amax(-1, keepdim=True)
            p = torch.exp(a - m)
            z = p.sum(-1, keepdim=True)
            p = p / z
            out[b] = torch.matmul(p, v).reshape(H, hd).to(kc.dtype)
            lse[b] = (m + torch.log(z)).reshape(H)
            if c["weights"]:
                w, nw = st["weights"][b], st["new_weights"][b]
                nw[:, :n] = w[:, :n]
                nw[:, j] = w[:, j] + p.sum(1)
        res = [out, lse, kc, vc]
        return res + [st["new_weights"]] if c["weights"] else res
    for b, n in enumerate(lengths):
        m = min(n, c["budget"])
        w = st["weights"][b, :, :n]
        at = torch.arange(n, device="cuda")
        always = (at < c["sinks"]) | (at >= n - c["recent"])
        key = torch.where(always, float("inf"), w) if n > m else w
        order = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :m]
        kept = torch.sort(order, dim=-1).values                       # [K, m]
        page, row = _rows(st, b, n)
        new = st["dst_page_table"][b].long()[at[:m] // ps]
        for h in range(K):
            for x in (kc, vc):
                x[new, h, at[:m] % ps] = x[page[kept[h]], h, row[kept[h]]]
        st["new_weights"][b] = 0
        st["new_weights"][b, :, :m] = torch.gather(w, 1, kept)
        st["kept"][b] = -1
        st["kept"][b, :, :m] = kept.int()
        st["new_lengths"][b] = m
    return [kc, vc, st["new_weights"], st["new_lengths"], st["kept"]]


# ---- the definition in 64 bits -------------------------------------------------------
def _mask64(S, length, window, sinks):
    i = torch.arange(S, device="cuda").view(S, 1)
    j = torch.arange(S, device="cuda").view(1, S)
    near = (i - j < window) if window else torch.ones_like(i - j, dtype=torch.bool)
    return (i >= j) & (near | (j < sinks)) & (i < length)


def _exact_seq(case, st):
    B, S, H, K, hd = case["B"], case["S"], case["heads"], case["kv_heads"], case["hd"]
    train = case["op"] == "train"
    f64 = lambda x: st[x].double()
    q, k, v = f64("q"), f64("k"), f64("v")
    out, lse = torch.zeros_like(q), torch.zeros(B, S, H, dtype=torch.float64, device="cuda")
    if train:
        do = f64("dout")
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b, length in enumerate(_lengths(case)):
        mask = _mask64(S, length, case["window"], case["sinks"])[:length, :length]
        for h in range(H):
            u = h * K // H
            qh, kh, vh = q[b, :length, h], k[b, :length, u], v[b, :length, u]
            logits = (qh @ kh.T) / hd ** 0.5
            logits[~mask] = -torch.inf
            L = torch.logsumexp(logits, dim=1)
            prob = (logits - L[:, None]).exp_()
            out[b, :length, h], lse[b, :length, h] = prob @ vh, L
            if train:
                g = do[b, :length, h]
                dv[b, :length, u] += prob.T @ g
                dprob = g @ vh.T
                dlog = prob * (dprob - (prob * dprob).sum(1, keepdim=True)) / hd ** 0.5
                dq[b, :length, h] = dlog @ kh
                dk[b, :length, u] += dlog.T @ qh
    return [out, lse, dq, dk, dv] if train else [out, lse]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("fwd", "train"):
        return _exact_seq(case, st)
    B, H, K, hd, ps = case["B"], case["heads"], case["kv_heads"], case["hd"], case["page"]
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    table = st["page_table"].tolist()

    def gather(cache, b, h, positions, tab=table):
        pages = torch.tensor([tab[b][p // ps] for p in positions], device="cuda")
        rows = torch.tensor([p % ps for p in positions], device="cuda")
        return cache[pages, h, rows], pages, rows

    if case["op"] == "append":
        for b, n in enumerate(_lengths(case)):
            t = min(n, case["tokens"])
            for cache, new in ((kc, st["k"]), (vc, st["v"])):
                _, pages, rows = gather(cache, b, 0, range(n - t, n))
                for h in range(K):
                    cache[pages, h, rows] = new[b, :t, h].double()
        return [kc, vc]
    if case["op"] == "decode":
        out = torch.zeros(B, H, hd, dtype=torch.float64, device="cuda")
        lse = torch.zeros(B, H, dtype=torch.float64, device="cuda")
        w = st["weights"].double() if case["weights"] else None
        if case["weights"]:   # nothing is written behind a sequence's end
            for b, n in enumerate(_lengths(case)):
                w[b, :, n:] = 0
        for b, n in enumerate(_lengths(case)):
            page, row = table[b][(n - 1) // ps], (n - 1) % ps
            kc[page, :, row], vc[page, :, row] = st["k_new"][b].double(), st["v_new"][b].double()
            see = [p for p in range(n) if not case["window"] or p >= n - case["window"] or p < case["sinks"]]
            at = torch.tensor(see, device="cuda")
            for u in range(K):
                keys, pages, rows = gather(kc, b, u, see) if u == 0 else (kc[pages, u, rows], pages, rows)
                heads = slice(u * (H // K), (u + 1) * (H // K))
                logits = st["q"][b, heads].double() @ keys.T / hd ** 0.5
                lse[b, heads] = torch.logsumexp(logits, 1)
                prob = torch.softmax(logits, 1)
                out[b, heads] = prob @ vc[pages, u, rows]
                if case["weights"]:
                    w[b, u, at] += prob.sum(0)
        return [out, lse, kc, vc, w] if case["weights"] else [out, lse, kc, vc]
    new_w = torch.zeros_like(st["weights"], dtype=torch.float64)
    kept = torch.full((B, K, case["budget"]), -1, dtype=torch.int32, device="cuda")
    new_len = []
    dst = st["dst_page_table"].tolist()
    for b, n in enumerate(_lengths(case)):
        m = min(n, case["budget"])
        new_len.append(m)
        weights = st["weights"][b].cpu().tolist()
        for u in range(K):
            if n <= case["budget"]:
                keep = list(range(n))
            else:
                first, last = case["sinks"], n - case["recent"]
                middle = sorted(range(first, last), key=lambda p: (-weights[u][p], p))
                keep = sorted([*range(first), *middle[:m - first - case["recent"]], *range(last, n)])
            for cache in (kc, vc):
                rows, _, _ = gather(cache, b, u, keep)
                _, pages, at = gather(cache, b, u, range(m), dst)
                cache[pages, u, at] = rows
            new_w[b, u, :m] = torch.tensor([weights[u][p] for p in keep], dtype=torch.float64)
            kept[b, u, :m] = torch.tensor(keep, dtype=torch.int32)
    return [kc, vc, new_w, torch.tensor(new_len, dtype=torch.int32, device="cuda"), kept]

"""Serving operators around an 8-bit paged kv cache: what they cost and what they compute.

Three operators of a decode or prompt step of top-k sparse multi-query attention:

  plan    block tables, sequence offsets, token positions and cache slots of a batch, made on the
          GPU from the requests' context and query lengths and a stack of free pages
  append  new kv rows written into an e4m3 paged cache with one power-of-two scale per page
          (keys = values, one kv head), a page's older rows rescaled when its scale grows
  attn    attention of H query heads per token over that cache: over the topk logical positions
          of a list (slots outside the request's length are masked), or, without a list, over
          every position up to the token's own; fp32 attention sink; bf16 O and log2 LSE

Cases are dicts of plain values; `run` computes a case in elementary torch operations, or, with
`own` set, through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # A continuous-batching decode step: 128 running requests, one new token each.
        {"name": "plan_decode_r128", "op": "plan", "R": 128, "ctx": 32768, "new": 1, "page": 64,
         "prompts": 0, "chunk": 0, "pad": 0},
        # A mixed step: 480 decoding requests and 32 prompt chunks of up to 512 tokens, page 16.
        {"name": "plan_mixed_r512", "op": "plan", "R": 512, "ctx": 8192, "new": 1, "page": 16,
         "prompts": 32, "chunk": 512, "pad": 77},
        # One decoded token of one request, D = 64: the smallest cache write there is.
        {"name": "append_t1_d64", "op": "append", "R": 1, "ctx": 128, "new": 1, "D": 64,
         "page": 16},
        # The decode batch's cache write.
        {"name": "append_t128_d512", "op": "append", "R": 128, "ctx": 2048, "new": 1, "D": 512,
         "page": 64},
        # Prompt rows of a few requests, ragged lengths.
        {"name": "append_t8192_d512", "op": "append", "R": 5, "ctx": 700, "new": 1638, "D": 512,
         "page": 64},
        # One request decoding alone: latency.
        {"name": "attn_t1_h128_k2048", "op": "attn", "R": 1, "q": 1, "ctx": 8192, "H": 128,
         "D": 512, "topk": 2048, "page": 64, "pad": 0},
        # The small configuration (16 heads of 64, 32 slots), one token of each of 128 requests.
        {"name": "attn_t128_h16_d64_k32", "op": "attn", "R": 128, "q": 1, "ctx": 512, "H": 16,
         "D": 64, "topk": 32, "page": 16, "pad": 0},
        # A decode batch with 64 heads and 512 slots, in a batch padded for a fixed-size graph.
        {"name": "attn_t250_h64_k512", "op": "attn", "R": 250, "q": 1, "ctx": 4096, "H": 64,
         "D": 512, "topk": 512, "page": 64, "pad": 6},
        # The decode batch of the 128-head configuration.
        {"name": "attn_t128_h128_k2048", "op": "attn", "R": 128, "q": 1, "ctx": 8192, "H": 128,
         "D": 512, "topk": 2048, "page": 64, "pad": 0},
        # A prompt chunk of four requests: early tokens see fewer positions than topk.
        {"name": "attn_t1024_h128_k2048", "op": "attn", "R": 4, "q": 256, "ctx": 4096, "H": 128,
         "D": 512, "topk": 2048, "page": 64, "pad": 0},
        # No index list: long contexts of uneven lengths, decoded together.
        {"name": "attn_dense_t16_h128", "op": "attn", "R": 16, "q": 1, "ctx": 32768, "H": 128,
         "D": 512, "topk": 0, "page": 64, "pad": 0},
        # No index list, odd sizes: 37 requests with 3 drafted tokens each, 48 heads of 64.
        {"name": "attn_dense_t111_h48_d64", "op": "attn", "R": 37, "q": 3, "ctx": 1111, "H": 48,
         "D": 64, "topk": 0, "page": 32, "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "dense"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        R = _log(rng, 1, 1024)
        return {"op": "plan", "R": R, "ctx": _log(rng, 1, 32768), "new": rng.choice([1, 1, 2, 4]),
                "page": page, "prompts": rng.randint(0, min(R, 16)), "chunk": _log(rng, 1, 512),
                "pad": _log(rng, 1, 200)}
    if op == "append":
        R = _log(rng, 1, 256)
        return {"op": "append", "R": R, "ctx": _log(rng, 1, 2048),
                "new": _log(rng, 1, max(1, 8192 // R)), "D": rng.choice([64, 512]), "page": page}
    D = rng.choice([64, 512, 512])
    H = rng.choice([1, 16, 24, 48, 64, 65, 100, 128])
    if op == "attn":
        R = _log(rng, 1, 256)
        q = rng.choice([1, 1, 2, 5]) if R > 8 else _log(rng, 1, 64)
        return {"op": "attn", "R": R, "q": q, "ctx": _log(rng, 1, 6000), "H": H, "D": D,
                "topk": _log(rng, 1, 2048 if R * q <= 512 else 1024), "page": page,
                "pad": rng.randint(0, 9)}
    R = _log(rng, 1, 24)
    return {"op": "attn", "R": R, "q": rng.choice([1, 1, 2, 4]), "ctx": _log(rng, 1, 8192),
            "H": H, "D": D, "topk": 0, "page": page, "pad": rng.randint(0, 5)}


def _lens(case):
    """(context, query) lengths of the requests: a golden-ratio spread of the context over
    [ctx/2, ctx] (from 0 up for the last eighth), so that the work does not depend on the seed."""
    ctx, qry = [], []
    R = case["R"]
    for r in range(R):
        f = (r * 0.6180339887498949) % 1.0
        c = case["ctx"] * (1.0 - 0.5 * f) if 8 * (r + 1) <= 7 * R or R == 1 else case["ctx"] * f
        ctx.append(int(c))
        if case["op"] == "attn":
            qry.append(case["q"])
        elif case["op"] == "append":
            qry.append(max(1, int(case["new"] * (1.0 - 0.5 * f))) if case["new"] > 8 else case["new"])
        else:
            n = case["new"]
            if r >= R - case["prompts"]:
                n = int(case["chunk"] * f)
            qry.append(n)
    return ctx, qry


def _pages(n, page):
    return -(-n // page)


def _slots(case, ctx, qry):
    """Valid (token, slot) pairs of an attention case."""
    n = 0
    for c, q in zip(ctx, qry):
        if case["topk"]:
            n += sum(min(case["topk"], c + i + 1) for i in range(q))
        else:
            n += sum(c + i + 1 for i in range(q))
    return n


def work(case):
    ctx, qry = _lens(case)
    T = sum(qry)
    if case["op"] == "plan":
        width = _pages(max(c + q for c, q in zip(ctx, qry)), case["page"])
        need = sum(_pages(c + q, case["page"]) - _pages(c, case["page"]) for c, q in zip(ctx, qry))
        T += case["pad"]
        return {"bytes": 4 * (2 * case["R"] + 2 * case["R"] * width + need + 2 * case["R"] + 3 + 3 * T),
                "flops": 0}
    if case["op"] == "append":
        return {"bytes": T * (3 * case["D"] + 4) + 8 * case["R"], "flops": 0}
    n = _slots(case, ctx, qry)
    rows = sum(min(c + q, _slots(case, [c], [q])) for c, q in zip(ctx, qry))
    H, D = case["H"], case["D"]
    pages = sum(_pages(c + q, case["page"]) for c, q in zip(ctx, qry))
    return {"bytes": T * H * D * 4 + T * H * 4 + H * 4 + rows * D + 4 * T * case["topk"] + 8 * pages,
            "flops": 4 * H * D * n}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _table(ctx_pages, width, n_pages, g):
    """Pages dealt to the requests in random order; the rest is the stack of free pages."""
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    k = torch.tensor(ctx_pages, device=DEV)
    first = torch.cumsum(k, 0) - k
    col = torch.arange(width, device=DEV)
    held = col[None, :] < k[:, None]
    at = (first[:, None] + col[None, :]).clamp(max=n_pages - 1)
    table = torch.where(held, perm[at], torch.full_like(perm[at], -1))
    used = sum(ctx_pages)
    return table.contiguous(), perm[used:].contiguous()


def _cache(n_pages, page, D, g):
    """A filled cache: rows N(0, 1) times a magnitude of the page, scales as the append leaves
    them (the smallest power of two that keeps the page's largest value within 448)."""
    mag = torch.exp2(torch.rand(n_pages, 1, 1, generator=g, device=DEV) * 3.0 - 2.0)
    x = torch.randn(n_pages, page, D, generator=g, device=DEV, dtype=torch.bfloat16).float() * mag
    m, e = torch.frexp(x.abs().amax(dim=(1, 2)))
    scale = torch.exp2((e - 9 + (m > 0.875)).float())
    return (x / scale[:, None, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    g = _gen(seed)
    ctx, qry = _lens(case)
    page, R, T = case["page"], case["R"], sum(qry)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    have = [_pages(c, page) for c in ctx]
    full = [_pages(c + q, page) for c, q in zip(ctx, qry)]
    width = max(full)
    if case["op"] == "plan":
        n_pages = sum(full) + R
        table, free = _table(have, width, n_pages, g)
        return {"case": dict(case), "context_lens": i32(ctx), "query_lens": i32(qry),
                "block_table": table, "free_pages": free, "free_count": i32([free.numel()]),
                "n_pages": n_pages, "max_tokens": T + case["pad"]}
    n_pages = sum(full) + 8
    table, _ = _table(full, width, n_pages, g)
    cache, scale = _cache(n_pages, page, case["D"], g)
    req = torch.repeat_interleave(torch.arange(R, device=DEV), i32(qry), output_size=T)
    start = torch.cumsum(i32(qry), 0) - i32(qry)
    pos = i32(ctx)[req] + torch.arange(T, device=DEV) - start[req]
    if case["op"] == "append":
        slot = table[req, (pos // page).long()].long() * page + pos % page
        new = torch.randn(T, case["D"], generator=g, device=DEV) * \
            torch.exp2(torch.rand(T, 1, generator=g, device=DEV) * 3.0 - 1.5)
        return {"case": dict(case), "kv_new": new.to(torch.bfloat16),
                "slot_mapping": slot.to(torch.int32), "kv_cache": cache, "kv_scales": scale}
    pad = case["pad"]
    H, D, K = case["H"], case["D"], case["topk"]
    seq = i32([c + q for c, q in zip(ctx, qry)])
    idx = None
    if K:
        L = max(ctx) + max(qry)
        keys = torch.rand(T, max(L, K), generator=g, device=DEV)
        keys = keys.masked_fill(torch.arange(max(L, K), device=DEV)[None, :] > pos[:, None], 2.0)
        val, idx = torch.topk(keys, K, dim=1, largest=False, sorted=True)  # the valid ones first
        idx = idx.to(torch.int32).masked_fill(val >= 2.0, -1)
        idx = torch.cat([idx, torch.full((pad, K), -1, dtype=torch.int32, device=DEV)])
    none = torch.full((pad,), -1, dtype=torch.int32, device=DEV)
    return {"case": dict(case), "q": torch.randn(T + pad, H, D, generator=g, device=DEV).to(torch.bfloat16),
            "kv_cache": cache, "kv_scales": scale,
            "attn_sink": torch.randn(H, generator=g, device=DEV), "block_table": table,
            "seq_lens": seq, "token_req": torch.cat([req.to(torch.int32), none]),
            "positions": torch.cat([pos.to(torch.int32), none]), "topk_idxs": idx,
            "longest": max(c + q for c, q in zip(ctx, qry))}


# ------------------------------------------------------------------------------------- plain
def _plan(s):
    page, N = s["case"]["page"], s["max_tokens"]
    ctx, qry = s["context_lens"].long(), s["query_lens"].long()
    R, width = s["block_table"].shape
    have, full = (ctx + page - 1) // page, (ctx + qry + page - 1) // page
    need = full - have
    first = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEV)[None, :]
    fresh = (col >= have[:, None]) & (col < full[:, None])
    nth = first[:, None] + col - have[:, None]
    count = s["free_count"].long()
    at = count - 1 - nth
    page_id = s["free_pages"][at.clamp(0, s["free_pages"].numel() - 1)]
    table = torch.where(fresh, torch.where(at >= 0, page_id, -1), s["block_table"])
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(qry, 0)])
    t = torch.arange(N, device=DEV)
    req = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = req < R
    r = req.clamp(max=R - 1)
    pos = ctx[r] + t - cu[r]
    slot = table[r, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    i32 = lambda v: v.to(torch.int32)  # noqa: E731
    return [table, i32(count - need.sum()), i32(ctx + qry), i32(cu), i32(torch.where(live, r, -1)),
            i32(torch.where(live, pos, -1)), i32(torch.where(live, slot, -1))]


def _append(s):
    cache, scale = s["kv_cache"], s["kv_scales"]
    n, page, D = cache.shape
    slot = s["slot_mapping"].long()
    at, off = slot // page, slot % page
    new = s["kv_new"].float()
    top = torch.zeros(n, device=DEV).scatter_reduce_(0, at, new.abs().amax(1), "amax")
    begins = torch.full((n,), page, device=DEV).scatter_reduce_(0, at, off, "amin")
    m, e = torch.frexp(top)
    want = torch.exp2(torch.where(top > 0, e - 9 + (m > 0.875), -60).clamp(min=-60).float())
    grown = torch.where(begins == page, scale, torch.where(begins == 0, want, torch.maximum(want, scale)))
    touched = torch.nonzero(begins < page)[:, 0]
    codes = cache.view(torch.uint8)
    old = codes[touched].view(torch.float8_e4m3fn).float() * (scale / grown)[touched][:, None, None]
    row = torch.arange(page, device=DEV)[None, :] < begins[touched][:, None]
    codes[touched] = torch.where(row[:, :, None], old.to(torch.float8_e4m3fn).view(torch.uint8), codes[touched])
    codes.view(-1, D)[slot] = (new / grown[at][:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(grown)
    return [cache, scale]


def _attn(s):
    cache, scale = s["kv_cache"], s["kv_scales"]
    page, D = cache.shape[1:]
    req = s["token_req"].long()
    live = req >= 0
    req = req.clamp(min=0)
    length = torch.where(live, s["seq_lens"][req], 0)[:, None]
    if s["topk_idxs"] is None:
        idx = torch.arange(s["longest"], device=DEV)[None, :].expand(req.numel(), -1)
        ok = (idx < length) & (idx <= s["positions"][:, None])
    else:
        idx = s["topk_idxs"].long()
        ok = (idx >= 0) & (idx < length)
    idx = torch.where(ok, idx, 0)
    pg = torch.where(ok, s["block_table"][req[:, None], idx // page].long(), 0)
    kv = cache.view(torch.uint8).view(-1, D)[pg * page + idx % page].view(torch.float8_e4m3fn).float()
    kv = kv * torch.where(ok, scale[pg], 0.0)[:, :, None]
    x = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * D ** -0.5
    x = torch.where(ok[:, None, :], x, -math.inf)
    sink = s["attn_sink"][None, :]
    top = torch.maximum(x.amax(2), sink)
    p = torch.exp(x - top[:, :, None])
    total = p.sum(2) + torch.exp(sink - top)
    o = torch.matmul(p, kv) / total[:, :, None]
    lse = (torch.log(total) + top) / math.log(2.0)
    return [torch.where(live[:, None, None], o, 0.0).to(torch.bfloat16),
            torch.where(live[:, None], lse, -math.inf)]


def run(state):
    op, s = state["case"]["op"], state
    if own:
        import bwd_sparse_mqa_gb300 as g
        if op == "plan":
            return list(g.paged_plan(s["context_lens"], s["query_lens"], s["block_table"], s["free_pages"],
                                     s["free_count"], s["case"]["page"], s["max_tokens"], s["n_pages"]))
        if op == "append":
            return list(g.paged_kv_append(s["kv_new"], s["slot_mapping"], s["kv_cache"], s["kv_scales"]))
        return list(g.sparse_mqa_paged_fwd(s["q"], s["kv_cache"], s["kv_scales"], s["attn_sink"],
                                           s["block_table"], s["seq_lens"], s["token_req"],
                                           positions=s["positions"], topk_idxs=s["topk_idxs"]))
    return {"plan": _plan, "append": _append, "attn": _attn}[op](s)


# ------------------------------------------------------------------------------------- 64 bits
def _exact_append(s, ctx, qry):
    """Request by request, page by page: each page's rows in real numbers, their scale the least
    power of two that holds them, each row rounded to e4m3 once the scale is known."""
    page, D = s["case"]["page"], s["case"]["D"]
    val = s["kv_cache"].view(torch.uint8).view(torch.float8_e4m3fn).double()
    scale = s["kv_scales"].double()
    new, slot, t = s["kv_new"].double(), s["slot_mapping"].tolist(), 0
    for c, q in zip(ctx, qry):
        end = t + q
        while t < end:
            pg, off = divmod(slot[t], page)
            k = min(page - off, end - t)
            rows = new[t:t + k]
            m = float(rows.abs().max())
            e = -60 if m == 0 else max(-60, math.ceil(math.log2(m / 448.0)))
            e -= e > -60 and m <= 448.0 * 2.0 ** (e - 1)
            sc = 2.0 ** e if off == 0 else max(2.0 ** e, float(scale[pg]))
            if off:
                kept = val[pg, :off] * float(scale[pg]) / sc
                val[pg, :off] = kept.to(torch.float8_e4m3fn).double()
            val[pg, off:off + k] = (rows / sc).to(torch.float8_e4m3fn).double()
            scale[pg] = sc
            t += k
    return [val, scale]


def _exact_attn(s):
    page, D = s["case"]["page"], s["case"]["D"]
    T, H = s["q"].shape[:2]
    o = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
    sink = s["attn_sink"].double()
    req, pos, seq = s["token_req"].tolist(), s["positions"].tolist(), s["seq_lens"].tolist()
    codes = s["kv_cache"].view(torch.uint8)
    for t in range(T):
        if req[t] < 0:
            continue
        n = min(seq[req[t]], pos[t] + 1)
        j = torch.arange(n, device=DEV) if s["topk_idxs"] is None else s["topk_idxs"][t].long()
        j = j[(j >= 0) & (j < seq[req[t]])]
        pg = s["block_table"][req[t], j // page].long()
        k = codes[pg, j % page].view(torch.float8_e4m3fn).double() * s["kv_scales"][pg].double()[:, None]
        z = torch.cat([s["q"][t].double() @ k.T / math.sqrt(D), sink[:, None]], 1)
        lse[t] = torch.logsumexp(z, 1) / math.log(2.0)
        o[t] = torch.softmax(z, 1)[:, :-1] @ k
    return [o, lse]


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    ctx, qry = _lens(case)
    return _exact_append(s, ctx, qry) if case["op"] == "append" else _exact_attn(s)

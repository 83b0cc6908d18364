"""Operators that choose what sparse MQA attends to, and their training: cost and results.

  append  new rows into the 8-bit paged cache with the position rotation applied on the way (kv rows
          of 512 or 64, index keys of 128)
  topk    the positions a token attends to: blocks of keys ranked by the lightning indexer's score
          sum_h w[h] ReLU(q[h] . k) (a block by its best visible row), for prompts and training
  paged   the same over index keys held in the 8-bit paged cache, for decoding and prompt chunks
  scores  the indexer's scores at given positions, and their gradients with respect to its queries,
          weights and keys

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
        # One decoded token's index key: the smallest write of a decode step.
        {"name": "append_t1_d128", "op": "append", "R": 1, "ctx": 128, "new": 1, "D": 128,
         "rope": 64, "offset": 0, "interleaved": False, "page": 64},
        # The decode batch's kv rows, the last 64 elements rotated in pairs.
        {"name": "append_t128_d512", "op": "append", "R": 128, "ctx": 2048, "new": 1, "D": 512,
         "rope": 64, "offset": 448, "interleaved": True, "page": 64},
        # Prompt rows of a few requests, ragged lengths.
        {"name": "append_t8192_d512", "op": "append", "R": 5, "ctx": 700, "new": 1638, "D": 512,
         "rope": 64, "offset": 448, "interleaved": True, "page": 64},
        # The small configuration: 128 tokens, 16 heads of 64, 32 positions each.
        {"name": "topk_s128_h16_d64_k32", "op": "topk", "B": 1, "S": 128, "S_kv": 128, "H": 16,
         "D": 64, "topk": 32, "block": 1, "recent": 0},
        # Two training sequences of 4096 with 512 positions per token.
        {"name": "topk_b2_s4096_h64_k512", "op": "topk", "B": 2, "S": 4096, "S_kv": 4096, "H": 64,
         "D": 128, "topk": 512, "block": 1, "recent": 64},
        # The indexer's workload: S = 8192, H = 64, D = 128, topk = 2048.
        {"name": "topk_s8192_h64_k2048", "op": "topk", "B": 1, "S": 8192, "S_kv": 8192, "H": 64,
         "D": 128, "topk": 2048, "block": 1, "recent": 0},
        # The last chunk of a long prompt, in blocks of 64 positions.
        {"name": "topk_s1000_kv32768_h64_b64", "op": "topk", "B": 1, "S": 1000, "S_kv": 32768,
         "H": 64, "D": 128, "topk": 2048, "block": 64, "recent": 64},
        # One request decoding alone in a long context: latency.
        {"name": "paged_t1_ctx32768", "op": "paged", "R": 1, "q": 1, "ctx": 32768, "H": 64,
         "D": 128, "topk": 2048, "block": 1, "recent": 0, "page": 64, "pad": 0},
        # A decode batch of long contexts, padded for a fixed-size graph.
        {"name": "paged_t128_ctx32768", "op": "paged", "R": 128, "q": 1, "ctx": 32768, "H": 64,
         "D": 128, "topk": 2048, "block": 1, "recent": 0, "page": 64, "pad": 3},
        # Prompt chunks of four requests.
        {"name": "paged_t1024_ctx8192", "op": "paged", "R": 4, "q": 256, "ctx": 8192, "H": 64,
         "D": 128, "topk": 2048, "block": 1, "recent": 128, "page": 64, "pad": 0},
        # The small configuration's scores, forward only.
        {"name": "scores_s128_h16_d64_k32", "op": "scores", "B": 1, "S": 128, "S_kv": 128, "H": 16,
         "D": 64, "topk": 32, "masked": 0.1, "grad": False},
        # A training step of the indexer: scores and all gradients at its workload's sizes.
        {"name": "scores_s8192_h64_k2048", "op": "scores", "B": 1, "S": 8192, "S_kv": 8192, "H": 64,
         "D": 128, "topk": 2048, "masked": 0.0, "grad": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "topk", "topk", "paged", "paged", "scores", "scores"])
    if op == "append":
        R = _log(rng, 1, 256)
        D = rng.choice([64, 128, 512])
        rope = rng.choice([r for r in (16, 32, 64, 128) if r <= D])
        return {"op": "append", "R": R, "ctx": _log(rng, 1, 2048),
                "new": _log(rng, 1, max(1, 8192 // R)), "D": D, "rope": rope,
                "offset": rng.choice([0, D - rope]), "interleaved": rng.random() < 0.5,
                "page": rng.choice([16, 32, 64, 128])}
    H = rng.choice([1, 4, 8, 16, 24, 32, 48, 64, 64, 65, 100, 128])
    D = rng.choice([64, 128, 128])
    if op == "scores":
        S, B = _log(rng, 1, 4096), rng.choice([1, 1, 2])
        topk = _log(rng, 1, min(2048, (1 << 29) // (B * S * H)))
        return {"op": "scores", "B": B, "S": S, "S_kv": S + _log(rng, 1, 4096) - 1, "H": H, "D": D,
                "topk": topk, "masked": rng.choice([0.0, 0.1, 0.5]) if S * topk >= 64 else 0.0,
                "grad": rng.random() < 0.7}
    block = rng.choice([1, 1, 1, 2, 8, 16, 32, 64, 128])

    def some(n):  # positions per token, of at most n: four blocks and half of them, or fewer
        b = min(block, 1 << max(0, (n // 8).bit_length() - 1))
        topk = b * _log(rng, 1, max(1, min(2048, n // 2) // b))
        return {"topk": topk, "block": b, "recent": rng.choice([0, 0, 1, topk // 4]) if topk >= 4 * b else 0}

    if op == "topk":
        S = _log(rng, 1, 3000)
        S_kv = S + _log(rng, 64, 6000)
        return {"op": "topk", "B": rng.choice([1, 1, 2, 3]), "S": S, "S_kv": S_kv, "H": H, "D": D, **some(S_kv)}
    R = _log(rng, 1, 128)
    ctx = _log(rng, 64, 32768 if R <= 16 else 12000)
    return {"op": "paged", "R": R, "q": rng.choice([1, 1, 2, 5]) if R > 8 else _log(rng, 1, 128),
            "ctx": ctx, "H": H, "D": D, **some(ctx), "page": rng.choice([16, 32, 64, 128]),
            "pad": rng.randint(0, 9)}


def _lens(case):
    """(context, new) lengths of the requests: a golden-ratio spread of the context over
    [ctx/2, ctx] (from 0 up for the last eighth), so that the work does not depend on the seed."""
    ctx, new = [], []
    R = case["R"]
    for r in range(R):
        f = (r * 0.6180339887498949) % 1.0
        c = case["ctx"] * (1.0 - 0.5 * f) if 8 * (r + 1) <= 7 * R or R == 1 else case["ctx"] * f
        ctx.append(int(c))
        n = case["q"] if case["op"] == "paged" else case["new"]
        new.append(max(1, int(n * (1.0 - 0.5 * f))) if case["op"] == "append" and n > 8 else n)
    return ctx, new


def _pages(n, page):
    return -(-n // page)


def _seen(case):
    """Visible keys of every token, and the keys the call reads: (list, rows)."""
    if case["op"] == "topk":
        n = [case["S_kv"] - case["S"] + s + 1 for s in range(case["S"])] * case["B"]
        return n, case["B"] * case["S_kv"]
    ctx, new = _lens(case)
    return [c + i + 1 for c, q in zip(ctx, new) for i in range(q)], sum(c + q for c, q in zip(ctx, new))


def work(case):
    H, D, op = case.get("H"), case["D"], case["op"]
    if op == "append":
        T = sum(_lens(case)[1])
        return {"bytes": T * (3 * D + 8 + 4 * case["rope"]) + 8 * case["R"], "flops": 3 * T * case["rope"]}
    if op == "scores":
        T = case["B"] * case["S"]
        slots = int(T * case["topk"] * (1.0 - case["masked"]))
        # Forward: queries, weights, keys, list in, scores out; with gradients, once more
        # all of them and their own in, three gradients out.
        io = T * H * D * 2 + 4 * T * H + case["B"] * case["S_kv"] * D * 2
        return {"bytes": io + 8 * T * case["topk"] + (io + 4 * T * case["topk"] if case["grad"] else 0),
                "flops": 2 * H * D * slots * (4 if case["grad"] else 1)}
    seen, rows = _seen(case)
    ranked = [n for n in seen if n > case["topk"]]           # the others take all they see
    io = len(ranked) * (2 * H * D + 4 * H) + 4 * len(seen) * case["topk"]
    per_row = 2 * D if op == "topk" else D
    if op == "paged":
        io += sum(8 * _pages(c + q, case["page"]) for c, q in zip(*_lens(case)))
    return {"bytes": io + (rows * per_row if ranked else 0), "flops": 2 * H * D * sum(ranked)}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _table(pages, width, n_pages, g):
    """Pages dealt to the requests in random order; -1 behind."""
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    k = torch.tensor(pages, device=DEV)
    first = torch.cumsum(k, 0) - k
    col = torch.arange(width, device=DEV)
    at = (first[:, None] + col[None, :]).clamp(max=n_pages - 1)
    return torch.where(col[None, :] < k[:, None], perm[at], torch.full_like(perm[at], -1)).contiguous()


def _cache(n_pages, page, D, g, spread):
    """A filled cache: rows N(0, 1) times a magnitude of the page, scales as the append leaves
    them (the smallest power of two that keeps the page's largest value within 448)."""
    mag = torch.exp2(torch.rand(n_pages, 1, 1, generator=g, device=DEV) * spread - spread / 2)
    x = torch.randn(n_pages, page, D, generator=g, device=DEV, dtype=torch.bfloat16).float() * mag
    m, e = torch.frexp(x.abs().amax(dim=(1, 2)))
    scale = torch.exp2((e - 9 + (m > 0.875)).float())
    return (x / scale[:, None, None]).to(torch.float8_e4m3fn), scale


def _cos_sin(n, rope):
    """[n, rope] fp32: cosines, then sines, of position * 10000^(-2 i / rope), angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(0, rope, 2, device=DEV, dtype=torch.float64) / rope)
    ang = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * freq[None, :]
    return torch.cat([torch.cos(ang), torch.sin(ang)], 1).float()


def prepare(case, seed):
    g = _gen(seed)
    op, D = case["op"], case["D"]
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if op in ("topk", "scores"):
        B, S, S_kv, H = case["B"], case["S"], case["S_kv"], case["H"]
        s = {"case": dict(case), "q": randn(B, S, H, D).to(torch.bfloat16),
             "w": randn(B, S, H) * (H * D) ** -0.5, "k": randn(B, S_kv, D).to(torch.bfloat16)}
        if op == "scores":
            K = case["topk"]
            idx = torch.randint(0, S_kv, (B, S, K), generator=g, device=DEV, dtype=torch.int32)
            out = torch.rand(B, S, K, generator=g, device=DEV) < case["masked"]
            s["idx"] = idx.masked_fill(out, -1)
            s["g"] = randn(B, S, K) / K
        return s
    ctx, new = _lens(case)
    page, R, T = case["page"], case["R"], sum(new)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    full = [_pages(c + q, page) for c, q in zip(ctx, new)]
    n_pages = sum(full) + 8
    table = _table(full, max(full), n_pages, g)
    cache, scale = _cache(n_pages, page, D, g, 3.0 if op == "append" else 1.0)
    req = torch.repeat_interleave(torch.arange(R, device=DEV), i32(new), output_size=T)
    start = torch.cumsum(i32(new), 0) - i32(new)
    pos = i32(ctx)[req] + torch.arange(T, device=DEV) - start[req]
    if op == "append":
        slot = table[req, (pos // page).long()].long() * page + pos % page
        rows = randn(T, D) * torch.exp2(torch.rand(T, 1, generator=g, device=DEV) * 3.0 - 1.5)
        return {"case": dict(case), "kv_new": rows.to(torch.bfloat16), "slot_mapping": slot.to(torch.int32),
                "kv_cache": cache, "kv_scales": scale, "positions": pos.to(torch.int32),
                "cos_sin": _cos_sin(max(c + q for c, q in zip(ctx, new)), case["rope"])}
    pad, H = case["pad"], case["H"]
    none = torch.full((pad,), -1, dtype=torch.int32, device=DEV)
    return {"case": dict(case), "q": randn(T + pad, H, D).to(torch.bfloat16),
            "w": randn(T + pad, H) * (H * D) ** -0.5, "k_cache": cache, "k_scales": scale,
            "block_table": table, "seq_lens": i32([c + q for c, q in zip(ctx, new)]),
            "token_req": torch.cat([req.to(torch.int32), none]),
            "positions": torch.cat([pos.to(torch.int32), none]),
            "spans": [(r, sum(new[:r]), q, c) for r, (c, q) in enumerate(zip(ctx, new))]}


# ------------------------------------------------------------------------------------- plain
def _append(s):
    c = s["case"]
    cache, scale = s["kv_cache"], s["kv_scales"]
    n, page, D = cache.shape
    slot = s["slot_mapping"].long()
    at, off = slot // page, slot % page
    new, half = s["kv_new"].float(), c["rope"] // 2
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = cs[:, :half], cs[:, half:]
    part = new[:, c["offset"]:c["offset"] + c["rope"]]
    x, y = (part[:, 0::2], part[:, 1::2]) if c["interleaved"] else (part[:, :half], part[:, half:])
    a, b = x * cos - y * sin, y * cos + x * sin
    part = torch.stack([a, b], 2).flatten(1) if c["interleaved"] else torch.cat([a, b], 1)
    new = torch.cat([new[:, :c["offset"]], part, new[:, c["offset"] + c["rope"]:]], 1)
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


def _choose(case, q, w, k, seen, out):
    """out [T, topk] for tokens q [T,H,D], w [T,H] that see the first seen [T] rows of k [n,D]:
    scores in 32 bits, those that may lie on either side of the border once more in 64."""
    n, bs, topk, recent = k.shape[0], case["block"], case["topk"], case["recent"]
    nb, kb = _pages(n, bs), case["topk"] // bs
    row = torch.arange(nb * bs, device=DEV)
    step = max(1, (1 << 29) // (q.shape[1] * max(n, 1)))
    length = k.norm(dim=1).max()
    for t0 in range(0, q.shape[0], step):
        t1 = min(t0 + step, q.shape[0])
        qt, wt, vis = q[t0:t1], w[t0:t1], seen[t0:t1, None]
        x = torch.matmul(qt.reshape(-1, qt.shape[2]), k.T).view(t1 - t0, -1, n).relu_()
        s = torch.bmm(wt[:, None, :], x)[:, 0]
        s = torch.nn.functional.pad(s, (0, nb * bs - n))
        s = torch.where(row < vis, s, -math.inf).view(t1 - t0, nb, bs).amax(2).double()
        s = torch.where(((row < vis) & (row >= vis - recent)).view(-1, nb, bs).any(2), math.inf, s)
        if kb < nb:
            border = torch.topk(s, kb, dim=1).values[:, -1:]
            near = 2.0 ** -15 * length * (wt.abs() * qt.norm(dim=2)).sum(1, keepdim=True)
            t, b = torch.nonzero((s - border).abs() <= near, as_tuple=True)
            for i in range(0, t.numel(), max(1, 4096 // bs)):
                ti, bi = t[i:i + max(1, 4096 // bs)], b[i:i + max(1, 4096 // bs)]
                j = bi[:, None] * bs + row[None, :bs]
                z = torch.bmm(qt[ti].double(), k[j.clamp(max=n - 1)].double().transpose(1, 2))
                z = torch.bmm(wt[ti].double()[:, None, :], z.relu_())[:, 0]
                s[ti, bi] = torch.where(j < vis[ti], z, -math.inf).amax(1)
            first = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :kb]
            took = torch.zeros_like(s, dtype=torch.bool).scatter_(1, first, True)
        else:
            took = torch.ones_like(s, dtype=torch.bool)
        took = took.repeat_interleave(bs, 1) & (row < vis)
        pos = torch.sort(torch.where(took, row, nb * bs), dim=1).values[:, :topk]
        out[t0:t1, :pos.shape[1]] = torch.where(pos < nb * bs, pos, -1).to(torch.int32)
    return out


def _topk(s):
    c = s["case"]
    out = torch.full((c["B"], c["S"], c["topk"]), -1, dtype=torch.int32, device=DEV)
    seen = torch.arange(c["S"], device=DEV) + c["S_kv"] - c["S"] + 1
    for b in range(c["B"]):
        _choose(c, s["q"][b].float(), s["w"][b], s["k"][b].float(), seen, out[b])
    return [out]


def _paged(s):
    c = s["case"]
    page, D = s["k_cache"].shape[1:]
    out = torch.full((s["q"].shape[0], c["topk"]), -1, dtype=torch.int32, device=DEV)
    codes = s["k_cache"].view(torch.uint8)
    for r, t0, q, ctx in s["spans"]:
        pg = s["block_table"][r, :_pages(ctx + q, page)].long()
        k = codes[pg].view(torch.float8_e4m3fn).float() * s["k_scales"][pg][:, None, None]
        _choose(c, s["q"][t0:t0 + q].float(), s["w"][t0:t0 + q], k.view(-1, D)[:ctx + q],
                s["positions"][t0:t0 + q].long() + 1, out[t0:t0 + q])
    return [out]


def _scores(s):
    c = s["case"]
    out = torch.empty_like(s["g"])
    dq, dw = torch.empty_like(s["q"]), torch.empty_like(s["w"])
    dk = torch.zeros(s["k"].shape, device=DEV)
    step = max(1, (1 << 27) // (c["topk"] * max(c["H"], c["D"])))
    for b in range(c["B"]):
        k = s["k"][b].float()
        for t in range(0, c["S"], step):
            at = slice(t, t + step)
            idx, w, q = s["idx"][b, at].long(), s["w"][b, at], s["q"][b, at].float()
            ok = (idx >= 0) & (idx < c["S_kv"])
            kj = k[idx.clamp(0, c["S_kv"] - 1)]                        # [t, topk, D]
            x = torch.bmm(q, kj.transpose(1, 2))                       # [t, H, topk]
            out[b, at] = torch.where(ok, torch.bmm(w[:, None, :], x.relu())[:, 0], -math.inf)
            if c["grad"]:
                g = torch.where(ok, s["g"][b, at], 0.0)
                dw[b, at] = torch.bmm(x.relu(), g[:, :, None])[:, :, 0]
                z = (x > 0) * g[:, None, :] * w[:, :, None]
                dq[b, at] = torch.bmm(z, kj).to(torch.bfloat16)
                dk[b].index_add_(0, idx.clamp(0, c["S_kv"] - 1).flatten(),
                                 torch.bmm(z.transpose(1, 2), q).flatten(0, 1))
    return [out, dq, dw, dk.to(torch.bfloat16)] if c["grad"] else [out]


def run(state):
    s, c = state, state["case"]
    if own:
        import bwd_sparse_mqa_gb300 as g
        if c["op"] == "append":
            return list(g.paged_kv_append(s["kv_new"], s["slot_mapping"], s["kv_cache"], s["kv_scales"],
                                          positions=s["positions"], cos_sin=s["cos_sin"],
                                          rope_offset=c["offset"], interleaved=c["interleaved"]))
        if c["op"] == "topk":
            return [g.indexer_topk(s["q"], s["w"], s["k"], c["topk"], block_size=c["block"],
                                   recent=c["recent"])]
        if c["op"] == "paged":
            return [g.paged_indexer_topk(s["q"], s["w"], s["k_cache"], s["k_scales"], s["block_table"],
                                         s["seq_lens"], s["token_req"], s["positions"], c["topk"],
                                         block_size=c["block"], recent=c["recent"])]
        if not c["grad"]:
            return [g.indexer_scores(s["q"], s["w"], s["k"], s["idx"])]
        q, w, k = (s[n].detach().requires_grad_() for n in ("q", "w", "k"))
        scores = g.indexer_scores(q, w, k, s["idx"])
        return [scores.detach(), *torch.autograd.grad(scores, (q, w, k), s["g"])]
    return {"append": _append, "topk": _topk, "paged": _paged, "scores": _scores}[c["op"]](s)


# ------------------------------------------------------------------------------------- 64 bits
def _exact_append(s, ctx, new):
    """Request by request, page by page: rows as complex numbers turned by their angle, a page's
    scale the least power of two that holds them, each row rounded to e4m3 once it is known."""
    c = s["case"]
    page = c["page"]
    val = s["kv_cache"].view(torch.uint8).view(torch.float8_e4m3fn).double()
    scale = s["kv_scales"].double()
    rows, slot, half = s["kv_new"].double(), s["slot_mapping"].tolist(), c["rope"] // 2
    turn = torch.view_as_complex(s["cos_sin"].double().view(-1, 2, half).transpose(1, 2).contiguous())
    turn = turn[s["positions"].long()]
    part = rows[:, c["offset"]:c["offset"] + c["rope"]]
    shape = (-1, half, 2) if c["interleaved"] else (-1, 2, half)
    pairs = part.reshape(shape) if c["interleaved"] else part.reshape(shape).transpose(1, 2)
    done = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    rows[:, c["offset"]:c["offset"] + c["rope"]] = (done if c["interleaved"] else done.transpose(1, 2)).reshape(len(slot), -1)
    t = 0
    for q in new:
        end = t + q
        while t < end:
            pg, off = divmod(slot[t], page)
            k = min(page - off, end - t)
            m = float(rows[t:t + k].abs().max())
            e = -60 if m == 0 else max(-60, math.ceil(math.log2(m / 448.0)))
            e -= e > -60 and m <= 448.0 * 2.0 ** (e - 1)
            sc = 2.0 ** e if off == 0 else max(2.0 ** e, float(scale[pg]))
            if off:
                val[pg, :off] = (val[pg, :off] * float(scale[pg]) / sc).to(torch.float8_e4m3fn).double()
            val[pg, off:off + k] = (rows[t:t + k] / sc).to(torch.float8_e4m3fn).double()
            scale[pg] = sc
            t += k
    return [val, scale]


def _exact_scores(s):
    """Token by token, head sums and gradients as matrix products over its valid slots."""
    c = s["case"]
    out = torch.full(s["g"].shape, -math.inf, dtype=torch.float64, device=DEV)
    dq, dw, dk = (torch.zeros(s[n].shape, dtype=torch.float64, device=DEV) for n in ("q", "w", "k"))
    for b in range(c["B"]):
        k = s["k"][b].double()
        for t in range(c["S"]):
            idx = s["idx"][b, t].long()
            ok = (idx >= 0) & (idx < c["S_kv"])
            kj = k[idx.clamp(0, c["S_kv"] - 1)] * ok[:, None]
            q, w = s["q"][b, t].double(), s["w"][b, t].double()
            act = (kj @ q.T).clamp(min=0)                              # [topk, H]
            out[b, t].copy_(torch.where(ok, act @ w, -math.inf))
            if c["grad"]:
                g = s["g"][b, t].double() * ok
                dw[b, t] = g @ act
                z = g[:, None] * ((act > 0) * w)
                dq[b, t] = z.T @ kj
                dk[b].index_add_(0, idx.clamp(0, c["S_kv"] - 1), z @ q)
    return [out, dq, dw, dk] if c["grad"] else [out]


def exact(case, seed):
    if case["op"] in ("topk", "paged"):
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_append(s, *_lens(case)) if case["op"] == "append" else _exact_scores(s)

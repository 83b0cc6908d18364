"""Plain 64-bit forms of the paged-cache operators, and their error bounds.

Bounds of the attention, element by element, for one token and head with
weights p_j = exp(x_j), l = sum p_j + exp(sink), and eps = 2^-24 (half a step
of fp32):
  logit   |dx_j| <= sm_scale (2^-22 max_d|q_d| + 2 D eps max_d|q_d|) sum_d|k_jd|
          (q as two e4m3 pieces of its scaled row leave at most 2^-22 of the
          row's largest value; the fp32 sum of D products adds the rest) +
          4 eps |x_j| (scale factors, and the running maximum's subtraction)
  weight  two e4m3 pieces of its value in fp16: 2^-4 of 2^-4 of the weight, and
          2^-11 for the step through fp16, relative; and 2^-14 of the token's
          largest weight (p_j s_j) where the second piece is subnormal: codes
          are multiples of 2^-9, so it is off by 2^-10 at most, and the largest
          weight's code is at least 2^(8 - 2 - 2) = 2^4 (m starts 2 above the
          first block's maximum, and weights are 2^-2 2^8 at m); 2^-21 for exp2
  O       2^-9 relative for its own rounding to bf16, the weights' error times
          |k_jd|, n eps for the fp32 sums
  lse     max_j |dx_j| / ln 2, exp2 and sums (2^-21 + n eps) / ln 2, and
          2^-22 (1 + |lse|) for its own log2 and rounding
"""
import math

import torch


def plan(ctx, qry, table, free, count, page, max_tokens, n_pages):
    """Python integers, request by request."""
    table = [list(r) for r in table]
    ctx, qry = [max(c, 0) for c in ctx], [max(q, 0) for q in qry]
    count = max(count, 0)
    left, taken = count, 0
    cu, req, pos, slot = [0], [], [], []
    for r, (c, q) in enumerate(zip(ctx, qry)):
        for col in range(-(-c // page), min(-(-(c + q) // page), len(table[r]))):
            table[r][col] = free[left - 1] if left > 0 else -1
            left -= left > 0
            taken += 1
        for p in range(c, c + q):
            pg = table[r][p // page] if p // page < len(table[r]) else -1
            req.append(r)
            pos.append(p)
            slot.append(pg * page + p % page if 0 <= pg < n_pages else -1)
        cu.append(cu[-1] + q)
    fill = lambda v: (v + [-1] * max_tokens)[:max_tokens]  # noqa: E731
    return (table, [count - taken], [c + q for c, q in zip(ctx, qry)], cu, fill(req), fill(pos),
            fill(slot))


def e4m3(x):
    """Nearest e4m3 value of float64 x (ties to even; |x| <= 448), by the format's definition."""
    mag = x.abs()
    e = torch.floor(torch.log2(torch.where(mag > 0, mag, torch.ones_like(mag)))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.sign(x) * torch.round(mag / step) * step


def append(new, slot, val, scale, page):
    """val [n_pages, page, D] (codes as float64), scale [n_pages] float64; returns new ones."""
    val, scale = val.clone(), scale.clone()
    n_pages, t, T = val.shape[0], 0, len(slot)
    while t < T:
        s = slot[t]
        if not 0 <= s < n_pages * page:
            t += 1
            continue
        pg, off = divmod(s, page)
        k = 1
        while t + k < T and slot[t + k] == s + k and off + k < page:
            k += 1
        x = new[t:t + k].double()
        fin = x[torch.isfinite(x)].abs()
        m = float(fin.max()) if fin.numel() else 0.0
        e = -60
        while m > 448.0 * 2.0 ** e:
            e += 1
        s1 = 2.0 ** e if off == 0 else max(2.0 ** e, float(scale[pg]))
        if off:
            val[pg, :off] = e4m3(val[pg, :off] * (float(scale[pg]) / s1))
        q = e4m3(torch.where(torch.isfinite(x), x, torch.zeros_like(x)) / s1)
        val[pg, off:off + k] = torch.where(torch.isfinite(x), q, torch.full_like(q, math.nan))
        scale[pg] = s1
        t += k
    return val, scale


def codes(kv_cache):
    """float8_e4m3fn -> float64 on the CPU."""
    return kv_cache.cpu().view(torch.uint8).view(torch.float8_e4m3fn).float().double()


def attn(q, val, scale, sink, table, seq, req, pos=None, idx=None, sm_scale=None):
    """(o, lse, bound of o, bound of lse), float64; val, scale as in append. Tokens of no
    request: zeros and -inf."""
    T, H, D = q.shape
    n_pages, page = val.shape[:2]
    R, W = table.shape
    sm = D ** -0.5 if sm_scale is None else sm_scale
    eps = 2.0 ** -24
    o = torch.zeros(T, H, D, dtype=torch.float64)
    bo = torch.zeros_like(o)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    bl = torch.zeros_like(lse)
    q, sink = q.double(), sink.double()
    for t in range(T):
        r = int(req[t])
        if not 0 <= r < R:
            continue
        n = int(seq[r])
        j = torch.arange(max(0, min(n, int(pos[t]) + 1))) if idx is None else idx[t].long()
        j = j[(j >= 0) & (j < n) & (j < W * page)]
        pg = table[r, j // page].long()
        j, pg = j[(pg >= 0) & (pg < n_pages)], pg[(pg >= 0) & (pg < n_pages)]
        c, s = val[pg, j % page], scale[pg]
        k = c * s[:, None]
        x = sm * q[t] @ k.T                                       # [H, n]
        z = torch.cat([x, sink[:, None]], 1)
        top = z.max(1, keepdim=True).values
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        p = torch.exp(x - top)
        l = p.sum(1, keepdim=True) + torch.exp(sink[:, None] - top)  # noqa: E741
        lse[t] = ((torch.log(l) + top) / math.log(2.0))[:, 0]
        if j.numel() == 0:
            bl[t] = 2.0 ** -22 * (1 + lse[t].abs())
            continue
        o[t] = p @ k / l
        qmax = q[t].abs().amax(1, keepdim=True)
        dx = (sm * (2.0 ** -22 + 2 * D * eps) * qmax * k.abs().sum(1)[None, :] + 4 * eps * x.abs())
        w = p * s
        rel = torch.expm1(dx) + 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -21 + j.numel() * eps
        bo[t] = (2.0 ** -9 * o[t].abs() + (rel * p) @ k.abs() / l
                 + 2.0 ** -14 * w.amax(1, keepdim=True) / l * c.abs().sum(0)[None, :]
                 + o[t].abs() * (torch.expm1(dx.amax(1, keepdim=True)) + 2.0 ** -21 + j.numel() * eps))
        bl[t] = (dx.amax(1) + 2.0 ** -21 + j.numel() * eps) / math.log(2.0) + 2.0 ** -22 * (1 + lse[t].abs())
    return o, lse, bo, bl


def check_attn(got, want):
    """Each element within its bound; NaN and infinities where the definition has them."""
    o, lse = (x.detach().cpu().double() for x in got)
    ro, rl, bo, bl = want
    for g, r, b, name in ((o, ro, bo, "o"), (lse, rl, bl, "lse")):
        assert torch.equal(torch.isnan(g), torch.isnan(r)), name
        inf = torch.isinf(r)
        assert torch.equal(g[inf], r[inf]), name
        ok = torch.isfinite(r)
        assert torch.isfinite(g[ok]).all(), name
        over = ((g - r).abs() - b)[ok]
        if over.numel():
            k = int(over.argmax())
            assert float(over.max()) <= 0, (f"{name}: off by {float((g - r).abs()[ok][k]):.3e}, "
                                            f"bound {float(b[ok][k]):.3e}")


def fill_cache(n_pages, page, D, seed, spread=0):
    """A cache whose every row is set, its pages' magnitudes 2^[-spread, spread]; codes and
    scales as the append leaves them. (kv_cache, kv_scales) on the CPU."""
    g = torch.Generator().manual_seed(seed)
    mag = torch.exp2(torch.randint(-spread, spread + 1, (n_pages, 1, 1), generator=g).double())
    x = (torch.randn(n_pages, page, D, generator=g).double() * mag).bfloat16()
    val, scale = append(x.reshape(-1, D), list(range(n_pages * page)),
                        torch.zeros(n_pages, page, D, dtype=torch.float64),
                        torch.ones(n_pages, dtype=torch.float64), page)
    return val.float().to(torch.float8_e4m3fn), scale.float()


def deal(lens, page, W, n_pages, seed):
    """A block table: each request's pages, in a seeded order; the rest -1."""
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), W), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(lens):
        k = -(-n // page)
        table[r, :k] = perm[at:at + k]
        at += k
    return table, perm[at:]

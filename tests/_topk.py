"""The indexer's selection in 64 bits: every choice of positions is a fact about real numbers, so
the GPU's lists are compared for equality.  (In fp64 a score is off by some 2^-45 of
sum |w||q||k|; inputs whose border is closer than that, but for exact ties, do not come up.)"""
import math

import torch


def scores(q, w, k):
    """[H,D], [H], [n,D] -> [n], float64; IEEE arithmetic for infinities and NaN in k."""
    x = k.double() @ q.double().T
    x = torch.where(torch.isnan(x), x, x.clamp(min=0))
    return x @ w.double()


def choose(s, topk, block=1, recent=0, there=None):
    """Positions (ascending, -1 behind) for scores s [n] of the rows a token sees; `there` [n]:
    rows on pages that exist."""
    n = s.numel()
    there = torch.ones(n, dtype=torch.bool, device=s.device) if there is None else there
    nb = -(-n // block)
    cls = torch.where(torch.isnan(s), 1, 2)
    cls[max(0, n - recent):] = 3 if recent else cls[max(0, n - recent):]
    cls = torch.where(there, cls, 0)
    val = torch.where(cls == 2, s + 0.0, -math.inf)
    pad = nb * block - n
    cls = torch.nn.functional.pad(cls, (0, pad)).view(nb, block)
    val = torch.nn.functional.pad(val, (0, pad), value=-math.inf).view(nb, block)
    bc, bv = cls.amax(1), val.amax(1)
    order = torch.sort(bv, descending=True, stable=True).indices
    order = order[torch.sort(bc[order], descending=True, stable=True).indices]
    took = order[bc[order] > 0][:topk // block].sort().values
    pos = (took[:, None] * block + torch.arange(block, device=s.device)).flatten()
    pos = pos[pos < n]
    pos = pos[there[pos]] if pos.numel() else pos
    return torch.nn.functional.pad(pos, (0, topk - pos.numel()), value=-1)


def flat(q, w, k, topk, block=1, recent=0, first=None):
    """indexer_topk."""
    B, S = q.shape[:2]
    S_kv = k.shape[1]
    first = S_kv - S if first is None else first
    out = torch.full((B, S, topk), -1, dtype=torch.int64, device=q.device)
    for b in range(B):
        for t in range(S):
            n = max(0, min(S_kv, first + t + 1))
            if n:
                out[b, t] = choose(scores(q[b, t], w[b, t], k[b, :n]), topk, block, recent)
    return out


def paged(q, w, val, scale, table, seq, req, pos, topk, block=1, recent=0, fill=None):
    """paged_indexer_topk; val [n_pages,page,D] float64 codes; rows of padding tokens: `fill`."""
    T = q.shape[0]
    n_pages, page, D = val.shape
    R, W = table.shape
    out = torch.full((T, topk), -1, dtype=torch.int64, device=q.device)
    if fill is not None:
        out.copy_(fill)
    for t in range(T):
        r = int(req[t])
        if not 0 <= r < R:
            continue
        n = min(int(seq[r]), W * page)
        if pos is not None:
            n = min(n, int(pos[t]) + 1)
        n = max(n, 0)
        out[t] = -1
        if n == 0:
            continue
        j = torch.arange(n, device=q.device)
        pg = table[r, j // page].long()
        there = (pg >= 0) & (pg < n_pages)
        pg = torch.where(there, pg, 0)
        k = val[pg, j % page] * scale[pg][:, None]
        out[t] = choose(scores(q[t], w[t], k), topk, block, recent, there)
    return out

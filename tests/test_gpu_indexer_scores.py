"""The indexer's scores at given positions and their gradients against 64-bit forms.

Bounds, element by element, with eps = 2^-24 (half a step of fp32):
  logit    x = q.k in the tensor core: |dx| <= (D + 16) eps |q||k| (each product may lose what
           lies 2^24 below its step's largest term, and up to 16 step sums are rounded)
  score    sum_h |w_h| (|dx| + (H / 4 + 4) eps |x|)
  dweights sum_j |g_j| |dx|, and (topk / 4 + 4) eps sum_j |g_j| |x|
  dq, dk   w g in bf16: 2^-8 of every term (a rounding is off by half a step, 2^-8 of the value at
           most), (n + 16) eps of their sum for n terms of an fp32 sum, 2^-8 for the
           result's own rounding, and the whole term where |x| <= |dx|: there either
           gate is right
"""
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import (_lib, indexer_scores, indexer_scores_bwd, indexer_scores_fwd,
                                  indexer_topk)
from bwd_sparse_mqa_gb300.api import device_status

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def _inputs(B, S, S_kv, H, D, topk, masked, seed, spread=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, S, H, D, generator=g)
    k = torch.randn(B, S_kv, D, generator=g)
    if spread:
        k = k * torch.exp2(torch.randint(-spread, spread + 1, (B, S_kv, 1), generator=g).float())
    w = torch.randn(B, S, H, generator=g) * (H * D) ** -0.5
    idx = torch.randint(0, S_kv, (B, S, topk), generator=g, dtype=torch.int32)
    out = torch.rand(B, S, topk, generator=g) < masked
    bad = torch.tensor([-1, S_kv, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[torch.randint(0, 4, (B, S, topk), generator=g)]
    idx = torch.where(out, bad, idx)
    gr = torch.randn(B, S, topk, generator=g) / topk
    return q.bfloat16(), w, k.bfloat16(), idx, gr


def _want(q, w, k, idx, gr):
    """(value, bound) of scores, dq, dw, dk."""
    B, S, H, D = q.shape
    S_kv, topk = k.shape[1], idx.shape[2]
    q, w, k, gr = q.double(), w.double(), k.double(), gr.double()
    sc = torch.full((B, S, topk), -math.inf, dtype=torch.float64)
    bs = torch.zeros_like(sc)
    dq, bq = torch.zeros_like(q), torch.zeros_like(q)
    dw, bw = torch.zeros_like(w), torch.zeros_like(w)
    dk, bk, nk = torch.zeros_like(k), torch.zeros_like(k), torch.zeros(B, S_kv, 1, dtype=torch.float64)
    for b in range(B):
        for t in range(S):
            i = idx[b, t].long()
            ok = (i >= 0) & (i < S_kv)
            j = i[ok]
            kj, g = k[b, j], gr[b, t][ok]
            x = q[b, t] @ kj.T                                          # [H, n]
            dx = (D + 16) * EPS * q[b, t].norm(dim=1)[:, None] * kj.norm(dim=1)[None, :]
            a = x.clamp(min=0)
            wa = w[b, t].abs()[:, None]
            sc[b, t, ok] = w[b, t] @ a
            bs[b, t, ok] = (wa * (dx + (H / 4 + 4) * EPS * a)).sum(0) + 2.0 ** -149
            dw[b, t] = a @ g
            bw[b, t] = (dx + (topk / 4 + 4) * EPS * a) @ g.abs() + 2.0 ** -149
            z = w[b, t][:, None] * g[None, :]
            gate, open_ = (x > 0).double(), (x.abs() <= dx).double()
            dq[b, t] = (z * gate) @ kj
            bq[b, t] = (z.abs() * (gate * (2.0 ** -8 + (topk + 16) * EPS) + open_)) @ kj.abs()
            dk[b].index_add_(0, j, (z * gate).T @ q[b, t])
            bk[b].index_add_(0, j, (z.abs() * (gate * (2.0 ** -8 + 2.0 ** -12) + open_)).T @ q[b, t].abs())
            nk[b].index_add_(0, j, torch.ones(j.numel(), 1, dtype=torch.float64))
    bq += 2.0 ** -8 * (dq.abs() + bq) + 2.0 ** -133
    # (An fp32 sum of nk terms: nk eps of their sizes' sum, of which bk holds 2^-8.)
    bk += nk * EPS * bk * 2.0 ** 8
    b32 = bk.clone() + 2.0 ** -149
    bk += 2.0 ** -8 * (dk.abs() + bk) + 2.0 ** -133
    return (sc, bs), (dq, bq), (dw, bw), (dk, bk), (dk, b32)


def _close(name, got, want):
    v, b = want
    g = got.detach().cpu().double()
    inf = torch.isinf(v)
    assert torch.equal(g[inf], v[inf]), name
    assert torch.isfinite(g[~inf]).all(), name
    over = ((g - v).abs() - b)[~inf]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{name}: over by {float(over.max()):.3e}"


CASES = [  # B, S, S_kv, H, D, topk, masked, spread
    (1, 1, 1, 1, 64, 1, 0.0, 0), (1, 3, 40, 16, 64, 32, 0.1, 0), (2, 9, 300, 64, 128, 150, 0.1, 3), (1, 5, 700, 128, 128, 513, 0.3, 0),
    (1, 4, 65, 65, 64, 64, 0.0, 2), (3, 2, 130, 24, 128, 129, 0.5, 0), (1, 2, 5000, 48, 64, 1000, 0.0, 0), (1, 6, 50, 100, 128, 255, 0.9, 1),
    (1, 2, 8, 33, 128, 300, 0.0, 0),
]


@pytest.mark.parametrize("case", CASES)
def test_scores_and_gradients(case):
    *shape, masked, spread = case
    x = _inputs(*shape, masked, 7 + shape[3], spread)
    c = [v.cuda() for v in x]
    want = _want(*x)
    _close("scores", indexer_scores_fwd(*c[:4], check_status=True), want[0])
    dq, dw, dk = indexer_scores_bwd(*c, check_status=True)
    for n, g, r in (("dq", dq, want[1]), ("dw", dw, want[2]), ("dk", dk, want[3])):
        _close(n, g, r)
    dq2, dw2, dk32 = indexer_scores_bwd(*c, return_dk_accum_dtype=True)
    assert torch.equal(dq2, dq) and torch.equal(dw2, dw) and dk32.dtype == torch.float32
    _close("dk32", dk32, want[4])


def test_no_valid_slot_and_bad_values_behind_masks():
    """Tokens without a valid slot give -inf and gradients of 0; NaN and infinities in key rows
    that no slot names, and in gradients of masked slots, reach nothing."""
    q, w, k, idx, gr = _inputs(1, 6, 90, 32, 128, 130, 0.3, 3)
    idx[0, 2] = -1
    idx[0, 4] = 90
    idx[(idx == 0) | (idx == 7)] = 5
    k[0, 0], k[0, 7] = math.nan, math.inf
    gr[(idx < 0) | (idx >= 90)] = math.nan
    clean = k.clone()
    clean[0, 0] = clean[0, 7] = 0
    want = _want(q, w, clean, idx, torch.nan_to_num(gr))
    c = [v.cuda() for v in (q, w, k, idx, gr)]
    _close("scores", indexer_scores_fwd(*c[:4]), want[0])
    got = indexer_scores_bwd(*c)
    for n, g, r in zip(("dq", "dw", "dk"), got, want[1:4]):
        _close(n, g, r)
    for t in (2, 4):
        assert got[0][0, t].eq(0).all() and got[1][0, t].eq(0).all()
    assert got[2][0, [0, 7]].eq(0).all() and device_status() == 0


def test_autograd_and_differences():
    """Gradients reach queries, weights and keys; the weights' against differences of the scores
    (linear in the weights: exact up to the scores' bound)."""
    q, w, k, idx, gr = [v.cuda() for v in _inputs(2, 5, 60, 16, 64, 40, 0.2, 5)]
    lq, lw, lk = (v.clone().requires_grad_() for v in (q, w, k))
    s = indexer_scores(lq, lw, lk, idx)
    assert s.requires_grad and s.dtype == torch.float32
    loss = (torch.where(torch.isfinite(s), s, 0.0) * gr).sum()
    dq, dw, dk = torch.autograd.grad(loss, (lq, lw, lk))
    want = indexer_scores_bwd(q, w, k, idx, gr)
    assert torch.equal(dq, want[0]) and torch.equal(dw, want[1]) and dk.dtype == torch.bfloat16
    assert float((dk.float() - want[2].float()).abs().max()) <= 2.0 ** -7 * float(dk.abs().max())
    f = lambda ww: (torch.where(torch.isfinite(s), indexer_scores_fwd(q, ww, k, idx), 0.0).double() * gr.double()).sum((1, 2))  # noqa: E731
    for h in (0, 7, 15):
        up, down = w.clone(), w.clone()
        up[:, 2, h] += 0.5
        down[:, 2, h] -= 0.5
        num = (f(up) - f(down)) / (up - down)[:, 2, h].double()
        scale = float((s[torch.isfinite(s)].detach().abs().max() + 1) * gr.abs().sum())
        assert float((num - dw[:, 2, h].double()).abs().max()) <= 2.0 ** -17 * scale


def test_differences_of_queries_and_keys():
    """One step along a direction: the scores' change is the gradient's, where no gate turns
    (the logits' signs are those of a constant added to both)."""
    B, S, S_kv, H, D, topk = 1, 4, 30, 8, 64, 25
    g = torch.Generator().manual_seed(9)
    q = (torch.rand(B, S, H, D, generator=g) + 0.5).bfloat16()
    k = (torch.rand(B, S_kv, D, generator=g) + 0.5).bfloat16()       # every logit > 0
    w = torch.randn(B, S, H, generator=g)
    idx = torch.randint(0, S_kv, (B, S, topk), generator=g, dtype=torch.int32)
    gr = torch.randn(B, S, topk, generator=g)
    q, w, k, idx, gr = (v.cuda() for v in (q, w, k, idx, gr))
    dq, _, dk = indexer_scores_bwd(q, w, k, idx, gr, return_dk_accum_dtype=True)
    q2 = (q.float() + 0.125).bfloat16()
    k2 = (k.float() + 0.125).bfloat16()
    total = lambda a, c: float((indexer_scores_fwd(a, w, c, idx).double() * gr.double()).sum())  # noqa: E731
    base = total(q, k)
    # Linear in q and in k: the change is gradient x step, with w g's 2^-8 and dq's own 2^-8.
    size = float(w.abs().sum() * gr.abs().sum() / (S * 1.0) * 0.125 * 1.5 * D)
    for new, grad, step in ((total(q2, k), dq, q2.double() - q.double()), (total(q, k2), dk, k2.double() - k.double())):
        assert abs((new - base) - float((grad.double() * step).sum())) <= 2.0 ** -7 * size


def test_many_calls_streams_and_capture():
    """Two streams at once, and a captured forward and backward replayed on new inputs."""
    xs = [[v.cuda() for v in _inputs(1, 40, 400, 64, 128, 300, 0.1, i)] for i in range(2)]
    ref = [(indexer_scores_fwd(*x[:4]), *indexer_scores_bwd(*x, return_dk_accum_dtype=True)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        out = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                out.append((indexer_scores_fwd(*x[:4]), *indexer_scores_bwd(*x, return_dk_accum_dtype=True)))
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert all(torch.equal(u, v) for u, v in zip(a[:3], b[:3]))
            assert float((a[3] - b[3]).abs().max()) <= 2.0 ** -18 * float(b[3].abs().max()) * 40
    buf = [v.clone() for v in xs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lq, lw, lk = (buf[i].detach().requires_grad_() for i in range(3))
        s = indexer_scores(lq, lw, lk, buf[3])
        grads = torch.autograd.grad(s, (lq, lw, lk), buf[4])
    for dst, src in zip(buf, xs[1]):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.detach(), ref[1][0]) and torch.equal(grads[0], ref[1][1]) and torch.equal(grads[1], ref[1][2])
    assert device_status() == 0


def test_no_second_derivative():
    """Refused, not left out."""
    q, w, k, idx, gr = (v.cuda() for v in _inputs(1, 4, 50, 16, 64, 10, 0.1, 2))
    leaves = [v.detach().requires_grad_() for v in (q, w, k)]
    s = indexer_scores(*leaves, idx)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(s, leaves, gr, create_graph=True, retain_graph=True)
    assert len(torch.autograd.grad(s, leaves, gr)) == 3


def test_calls_from_threads_that_made_no_cuda_call():
    """As autograd's are: the calls make the device's context their own."""
    import threading
    x = [v.cuda() for v in _inputs(1, 6, 100, 16, 64, 20, 0.1, 4)]
    want = indexer_scores_fwd(*x[:4]), *indexer_scores_bwd(*x), indexer_topk(*x[:3], 5)
    for i, call in enumerate((lambda: (indexer_scores_bwd(*x)[0], 1), lambda: (indexer_topk(*x[:3], 5), 4), lambda: (indexer_scores_fwd(*x[:4]), 0))):
        got = []
        th = threading.Thread(target=lambda: got.append(call()))
        th.start()
        th.join()
        torch.cuda.synchronize()
        assert got and torch.equal(got[0][0], want[got[0][1]]), i


def test_bounded_wait_runs_out():
    lib = _lib.load()
    x = [v.cuda() for v in _inputs(1, 4, 200, 16, 128, 300, 0.0, 1)]
    old = lib.smqa_set_wait_limit_ns(50_000_000)
    try:
        for call in (lambda: indexer_scores_fwd(*x[:4], check_status=True), lambda: indexer_scores_bwd(*x, check_status=True)):
            lib.smqa_debug_stall(1)
            with pytest.raises(_lib.SMQAError):
                call()
            lib.smqa_debug_stall(-1)
            assert device_status(clear=True) == _lib.SMQA_ERR_DEVICE_TIMEOUT
            call()
    finally:
        lib.smqa_debug_stall(-1)
        lib.smqa_set_wait_limit_ns(0 if old == 4_000_000_000 else old)
        device_status(clear=True)


def test_refusals():
    q, w, k, idx, gr = [v.cuda() for v in _inputs(1, 3, 20, 16, 64, 8, 0.0, 1)]
    for bad in ((q[:, :2].contiguous(), w, k, idx), (q, w[:, :, :3].contiguous(), k, idx), (q, w, k[:, :, :32].contiguous(), idx),
                (q, w, k, idx[:, :2].contiguous()), (q.transpose(1, 2), w, k, idx), (q.cpu(), w, k, idx), (q, w, k, idx[0])):
        with pytest.raises(ValueError):
            indexer_scores_fwd(*bad)
    for bad in ((q.float(), w, k, idx), (q, w.double(), k, idx), (q, w, k, idx.long())):
        with pytest.raises(TypeError):
            indexer_scores_fwd(*bad)
    with pytest.raises(ValueError):
        indexer_scores_bwd(q, w, k, idx, gr[:, :, :4])
    with pytest.raises(TypeError):
        indexer_scores_bwd(q, w, k, idx, gr.double())
    with pytest.raises(_lib.SMQAError):
        indexer_scores_fwd(q[..., :32].contiguous(), w, k[..., :32].contiguous(), idx)
    with pytest.raises(_lib.SMQAError):
        indexer_scores_fwd(q, w, k, idx[:, :, :0].contiguous())


def test_training_step_with_the_selection():
    """Choose, score what was chosen, and learn: the chosen positions' scores are the best ones."""
    q, w, k, _, _ = [v.cuda() for v in _inputs(1, 50, 50, 16, 64, 8, 0.0, 2)]
    idx = indexer_topk(q, w, k, 12)
    lq, lw, lk = (v.clone().requires_grad_() for v in (q, w, k))
    s = indexer_scores(lq, lw, lk, idx)
    assert torch.equal(torch.isinf(s), idx < 0)
    every = torch.arange(50, dtype=torch.int32, device="cuda").expand(1, 50, 50).contiguous()
    full = indexer_scores_fwd(q, w, k, every)
    full = torch.where(torch.arange(50, device="cuda")[None, None] <= torch.arange(50, device="cuda")[None, :, None], full, -math.inf)
    best = torch.sort(full, dim=2, descending=True).values[:, :, :12]
    mine = torch.sort(s.detach(), dim=2, descending=True).values
    assert float((best - mine)[torch.isfinite(best)].abs().max()) <= 2.0 ** -17 * float(best[torch.isfinite(best)].abs().max() + 1)
    target = torch.softmax(torch.randn_like(s).masked_fill(torch.isinf(s), -math.inf), 2)
    loss = torch.nn.functional.kl_div(torch.log_softmax(s, 2).masked_fill(torch.isinf(s), 0.0), target, reduction="sum")
    loss.backward()
    for v in (lq, lw, lk):
        assert torch.isfinite(v.grad).all() and v.grad.abs().max() > 0

"""The attention over the 8-bit paged cache at the ends of its number range."""
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import sparse_mqa_paged_fwd
from tests import _paged as ref
from tests.test_gpu_paged_weights import attn64, call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [-101, -100, -99, 0, 124, 125, 126, 127])
@pytest.mark.parametrize("D", [64, 512])
def test_query_rows_up_to_the_largest(D, power):
    """A row's largest value in [2^power, 2^(power + 1)), the softmax scale (or the pages') such
    that the logits are moderate. q.c stays below 2^128: one element of q meets codes up to 1."""
    page, n, H = 16, 200, 6
    g = torch.Generator().manual_seed(D + power)
    n_pages = -(-n // page)
    big = power > 0
    scale = torch.full((n_pages,), 2.0 ** (-60 if big else 100 if power < -50 else 0), dtype=torch.float64)
    val = ref.e4m3(torch.randn(n_pages, page, D, generator=g).double().clamp(-2, 2) / 2)
    sm = 2.0 ** -66 if big else 1.0
    q = torch.zeros(H, D)
    q[torch.arange(H), torch.arange(H) * 7 + 3] = 2.0 ** power * torch.tensor([1.0, 1.5, -1.984375, 1.0, -1.0, 1.25])
    q = q.bfloat16()
    q[5, 40] = q[5, 38] * 2.0 ** -9                        # (two pieces: the finer one counts)
    sink, pos = torch.zeros(H), torch.arange(n)
    table = torch.arange(n_pages, dtype=torch.int32)[None].contiguous()
    got = call(q, val, scale, table, sink, n, sm=sm)
    o, b, lse = attn64(q, val, scale, sink, pos // page, pos % page, sm)
    over = (got[0].cpu().double() - o).abs() - b
    assert float(over.max()) <= 0, f"o: {float(over.max()):.3e} beyond its bound"
    assert float((got[1].cpu().double() - lse).abs().max()) <= 1e-4


@pytest.mark.parametrize("power", [-104, -110, -115, -119, -120, -124])
@pytest.mark.parametrize("D", [64, 512])
def test_query_rows_down_to_the_smallest(D, power):
    """Rows of q that are as small as bf16's normal numbers, over pages of scales up to 2^120: q's
    pieces hold a row down to 2^-22 of its largest value, or of 2^-119."""
    page, n, H = 16, 200, 6
    g = torch.Generator().manual_seed(D - power)
    n_pages = -(-n // page)
    scale = torch.full((n_pages,), 2.0 ** min(-power, 120), dtype=torch.float64)
    val = ref.e4m3(torch.randn(n_pages, page, D, generator=g).double().clamp(-3, 3) * 16)
    q = (torch.randn(H, D, generator=g).clamp(-2, 2) / 2 * 2.0 ** power).bfloat16()
    q[0] = 0
    sink, pos = torch.zeros(H), torch.arange(n)
    table = torch.arange(n_pages, dtype=torch.int32)[None].contiguous()
    got = call(q, val, scale, table, sink, n, sm=1.0 / 64)
    o, b, lse = attn64(q, val, scale, sink, pos // page, pos % page, 1.0 / 64)
    # q's own floor, 2^-22 of 2^-119, in the logits and so in the weights and l
    low = (2.0 ** -141 * (val * scale[:, None, None]).abs().sum(2).max() / 64).item()
    over = (got[0].cpu().double() - o).abs() - b - 2 * low * (val * scale[:, None, None]).abs().max()
    assert float(over.max()) <= 0, f"o: {float(over.max()):.3e} beyond its bound"
    assert float((got[1].cpu().double() - lse).abs().max()) <= 1e-4 + 2 * low


@pytest.mark.parametrize("low,high", [(-60, 40), (-60, 0), (20, 120), (-30, 70)])
@pytest.mark.parametrize("page", [16, 64])
def test_page_scales_as_far_apart_as_stated(low, high, page):
    """Pages of all zeros, or nearly, beside pages 2^100 above them whose rows are orthogonal to
    q: every position counts in l."""
    D, H, n_pages = 64, 16, 12
    g = torch.Generator().manual_seed(page + high)
    n = n_pages * page
    val = ref.e4m3(torch.randn(n_pages, page, D, generator=g).double().clamp(-3, 3) * 64)
    val[:, :, ::2] = 0
    scale = torch.where(torch.arange(n_pages) % 2 == 0, 2.0 ** low, 2.0 ** high).double()
    val[0] = 0
    q = torch.randn(H, D, generator=g)
    q[:, 1::2] = 0
    q = q.bfloat16()
    sink, pos = torch.full((H,), 3.0), torch.arange(n)
    table = torch.arange(n_pages, dtype=torch.int32)[None].contiguous()
    for idx in (None, torch.randperm(n, generator=g)):
        at = pos if idx is None else idx
        got = call(q, val, scale, table, sink, n, idx)
        o, b, lse = attn64(q, val, scale, sink, at // page, at % page, D ** -0.5)
        assert torch.allclose(lse, torch.full((H,), math.log2(n + math.exp(3.0))).double())
        # lse: sums of n terms, and top = log2 of the largest scale at most, in fp32
        assert float((got[1].cpu().double() - lse).abs().max()) <= 2.0 ** -14
        assert float(((got[0].cpu().double() - o).abs() - b).max()) <= 0


@pytest.mark.parametrize("topk", [0, 100, 8000])
def test_a_nan_sink_reaches_its_head(topk):
    """A NaN sink makes its head's O and LSE NaN, in tokens that attend to something, to nothing,
    whole or split, and leaves the other heads alone."""
    D, page, n = 64, 16, 9000 if topk != 100 else 60
    cache, scale = ref.fill_cache(-(-n // page), page, D, 3)
    table = torch.arange(cache.shape[0], dtype=torch.int32)[None].contiguous()
    g = torch.Generator().manual_seed(topk)
    q = torch.randn(2, 3, D, generator=g).bfloat16()
    sink = torch.tensor([0.5, math.nan, -math.inf])
    pos = torch.tensor([n - 1, -1], dtype=torch.int32)
    idx = None
    if topk:
        idx = torch.full((2, topk), -1, dtype=torch.int32)
        idx[0, :min(topk, n)] = torch.randperm(n, generator=g)[:min(topk, n)].int()
    got = sparse_mqa_paged_fwd(q.cuda(), cache.cuda(), scale.cuda(), sink.cuda(), table.cuda(),
                               torch.tensor([n], dtype=torch.int32, device="cuda"),
                               torch.zeros(2, dtype=torch.int32, device="cuda"), pos.cuda(),
                               None if idx is None else idx.cuda(), check_status=True)
    want = ref.attn(q, ref.codes(cache), scale.double(), torch.where(sink.isnan(), 0.0, sink), table, [n], [0, 0],
                    pos.tolist(), idx)
    for w in want:
        w[:, 1] = math.nan
    ref.check_attn(got, want)

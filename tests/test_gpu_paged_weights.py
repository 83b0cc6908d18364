"""The weights of the attention over the 8-bit paged cache, at the distributions
where few positions hold much of the weight and many share the rest: O against
64 bits, element by element, within bounds that do not grow with the number of
slots a token sees.

Bound of O for one token and head, with w_j = p_j s_j (p_j = exp(x_j), s_j the
scale of the position's page, c_j its codes) and l = sum p_j + exp(sink):
  a weight is held as two e4m3 pieces of its value in fp16, in units that go by
  the largest w of its group (32 slots in a row, of the list or of positions):
  relative 2^-4 of 2^-4 and 2^-11 for fp16, or, where the pieces are subnormal,
  2^-23 of a unit of which the group's largest is at least one half, and 2^-25
  for a subnormal fp16: (2^-8 + 2^-11) w_j + (2^-22 + 2^-24) max_group w;
  2^-21 for exp2, expm1(dx) for the logit (as in tests/_paged.py, but that its
  fp32 sum is off by 2 D 2^-24 of the sum of its products' magnitudes, and that
  zeros of q are held as they are: neither piece of them has a value), n 2^-26 for the
  tensor core's fp32 sums (an addition per 32 slots and piece, each off by 2^-23
  at most), all times |k_jd|; O's scale by l (the same dx, 2^-21), 2^-9 for
  its rounding to bf16, and 2^-126, below which neither it nor fp32 has normal
  numbers (weights e^-250 of the largest give an O of 10^-110: it is 0).
"""
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import sparse_mqa_fwd_interface, sparse_mqa_paged_fwd
from bwd_sparse_mqa_gb300.api import device_status
from tests import _paged as ref

GROUP = 32


def attn64(q, val, scale, sink, page_of, row_of, sm):
    """(o, bound of o, lse) of one token whose valid slots are rows (page_of, row_of), -1:
    masked; q [H, D]."""
    live = page_of >= 0
    s = torch.where(live, scale[page_of.clamp(min=0)], 0.0)
    c = val[page_of.clamp(min=0), row_of] * live[:, None]
    k = c * s[:, None]
    q = q.double()
    x = (sm * q @ k.T).masked_fill(~live[None, :], -math.inf)
    top = torch.maximum(x.max(1).values, sink.double())[:, None]
    p = torch.exp(x - top)
    l = p.sum(1, keepdim=True) + torch.exp(sink.double()[:, None] - top)  # noqa: E741
    o = p @ k / l
    n, D, eps = int(live.sum()), q.shape[1], 2.0 ** -24
    dx = (sm * (2.0 ** -22 * q.abs().amax(1, keepdim=True) * ((q != 0).double() @ k.abs().T) +
                2 * D * eps * q.abs() @ k.abs().T) + 4 * eps * x.abs().masked_fill(~live[None, :], 0.0))
    rel = torch.expm1(dx) + 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -21 + n * 2.0 ** -26
    w = p * s
    pad = -len(s) % GROUP
    floor = torch.nn.functional.pad(w, (0, pad)).unflatten(1, (-1, GROUP)).amax(2)
    mass = torch.nn.functional.pad(c.abs(), (0, 0, 0, pad)).unflatten(0, (-1, GROUP)).sum(1)
    b = (2.0 ** -126 + 2.0 ** -9 * o.abs() + (rel * p) @ k.abs() / l + (2.0 ** -22 + 2.0 ** -24) * floor @ mass / l
         + o.abs() * (torch.expm1(dx.amax(1, keepdim=True)) + 2.0 ** -21 + n * 2.0 ** -26))
    return o, b, ((torch.log(l) + top) / math.log(2.0))[:, 0]


def check(got, want):
    o, (r, b, lse) = got[0].cpu().double(), want
    over = (o - r).abs() - b
    worst = int(over.argmax())
    assert float(over.max()) <= 0, (f"o: off by {float((o - r).abs().flatten()[worst]):.3e}, "
                                    f"bound {float(b.flatten()[worst]):.3e}")
    # A row's error against its norm, whatever the number of slots.
    err = (o - r).norm(dim=1) / r.norm(dim=1)
    assert float(err.max()) <= 2.0 ** -7, f"o: off by {float(err.max()):.3e} of its norm"
    assert float((got[1].cpu().double() - lse).abs().max()) <= 2.0 ** -14 * (1 + float(lse.abs().max()))


def heavy_tail(n, D, H, page, seed, mean=1.0):
    """One request of n positions: rows of deviation 1 about a common mean, flat logits but for
    two positions, 5 and n - 100; heads in turn see one of them 8, 10, 12 or 14 nats above the
    rest, the later half of the heads with logits of deviation 1/4 besides."""
    g = torch.Generator().manual_seed(seed)
    rows = mean + torch.randn(n, D, generator=g)
    rows[:, :2] = 0
    rows[5, 0] = rows[n - 100, 1] = 4.0
    n_pages = -(-n // page) + 2
    table, _ = ref.deal([n], page, n_pages, n_pages, seed)
    pos = torch.arange(n)
    pg = table[0, pos // page].long()
    val, scale = ref.append(rows.bfloat16(), (pg * page + pos % page).tolist(),
                            torch.zeros(n_pages, page, D, dtype=torch.float64),
                            torch.ones(n_pages, dtype=torch.float64), page)
    q = torch.zeros(H, D)
    q[H // 2:, 2:] = 0.25 * torch.randn(H - H // 2, D - 2, generator=g)
    q[:, 2:] -= q[:, 2:].mean(1, keepdim=True)           # (the common mean leaves the logits alone)
    gap = torch.tensor([8.0, 10.0, 12.0, 14.0])[torch.arange(H) % 4]
    q[torch.arange(H), (torch.arange(H) // 4) % 2] = gap / 4.0 * D ** 0.5
    return q.bfloat16(), val, scale, table, pg, pos


def call(q, val, scale, table, sink, n, idx=None, sm=None):
    got = sparse_mqa_paged_fwd(q[None].cuda(), val.float().to(torch.float8_e4m3fn).cuda(), scale.float().cuda(),
                               sink.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                               torch.zeros(1, dtype=torch.int32, device="cuda"),
                               torch.tensor([n - 1], dtype=torch.int32, device="cuda"),
                               None if idx is None else idx[None].to(torch.int32).cuda(), sm_scale=sm)
    assert device_status() == 0
    return got[0][0], got[1][0]


@pytest.mark.gpu
@pytest.mark.parametrize("D,page", [(512, 64), (64, 16)])
@pytest.mark.parametrize("n", [1000, 2048, 8192, 32768])
def test_heavy_position_over_a_flat_rest(n, D, page):
    q, val, scale, table, pg, pos = heavy_tail(n, D, 48, page, n + D)
    sink = torch.full((48,), -1.0)
    got = call(q, val, scale, table, sink, n)
    check(got, attn64(q, val, scale, sink, pg, pos % page, D ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("D,H", [(512, 128), (64, 16)])
@pytest.mark.parametrize("n,topk", [(2048, 2048), (4000, 2048), (8192, 8192)])
def test_heavy_position_in_a_list(n, topk, D, H):
    """Both heavy positions listed, in some order among the others, a tenth of them masked."""
    q, val, scale, table, pg, pos = heavy_tail(n, D, H, 32, n + topk + D)
    g = torch.Generator().manual_seed(topk)
    idx = torch.randperm(n, generator=g)[:topk]
    idx[torch.rand(topk, generator=g) < 0.1] = -1
    at = torch.randperm(topk, generator=g)[:2]
    for a, heavy in zip(at.tolist(), (5, n - 100)):
        idx[idx == heavy] = -1
        idx[a] = heavy
    sink = torch.zeros(H)
    got = call(q, val, scale, table, sink, n, idx)
    safe = idx.clamp(min=0)
    check(got, attn64(q, val, scale, sink, torch.where(idx < 0, -1, pg[safe]), safe % 32, D ** -0.5))


@pytest.mark.gpu
def test_heavy_position_next_to_the_contiguous_forward():
    """e4m3 codes times a power of two are exact in bf16: the bf16 forward on the same rows."""
    n, D, H = 2048, 512, 64
    q, val, scale, table, pg, pos = heavy_tail(n, D, H, 64, 7)
    sink = torch.zeros(H)
    idx = torch.randperm(n, generator=torch.Generator().manual_seed(1))
    o, lse = call(q, val, scale, table, sink, n, idx)
    rows = (val * scale[:, None, None])[pg, pos % 64].bfloat16()
    o2, lse2 = sparse_mqa_fwd_interface(q[None, None].cuda(), rows[None].cuda(), sink.cuda(),
                                        idx[None, None].to(torch.int32).cuda())
    err = (o.float() - o2[0, 0].float()).norm(dim=1) / o2[0, 0].float().norm(dim=1)
    assert float(err.max()) <= 2.0 ** -7 and float((lse - lse2[0, 0]).abs().max()) <= 1e-3


@pytest.mark.gpu
@pytest.mark.parametrize("power", [0, 10, 12, 14])
def test_equal_weights_over_pages_of_unlike_scale(power):
    """Every other page holds one row 2^power above the rest, which the list leaves out: all
    listed rows have the same logit and like values, and scales up to 2^power apart."""
    D, page, H, n_pages = 512, 16, 16, 40
    g = torch.Generator().manual_seed(power)
    rows = (1.0 + 0.3 * torch.randn(n_pages * page, D, generator=g))
    rows[::2 * page] *= 2.0 ** power
    val, scale = ref.append(rows.bfloat16(), list(range(n_pages * page)),
                            torch.zeros(n_pages, page, D, dtype=torch.float64),
                            torch.ones(n_pages, dtype=torch.float64), page)
    idx = torch.randperm(n_pages * page, generator=g)
    idx = idx[idx % (2 * page) != 0]
    table = torch.arange(n_pages, dtype=torch.int32)[None].contiguous()
    q, sink = torch.zeros(H, D).bfloat16(), torch.full((H,), -2.0)
    got = call(q, val, scale, table, sink, n_pages * page, idx)
    check(got, attn64(q, val, scale, sink, idx // page, idx % page, D ** -0.5))


@pytest.mark.gpu
def test_weights_of_growing_and_falling_logits():
    """Logits that climb by 60 nats over the positions, and fall by as much: the sums' unit
    moves with them, and what came before is not lost."""
    n, D, page, H = 3000, 64, 64, 8
    g = torch.Generator().manual_seed(3)
    rows = 1.0 + torch.randn(n, D, generator=g)
    rows[:, 0] = torch.linspace(-4, 4, n)
    rows[:, 1] = 0
    rows[n // 2, 1] = 4.0
    n_pages = -(-n // page)
    val, scale = ref.append(rows.bfloat16(), list(range(n)), torch.zeros(n_pages, page, D, dtype=torch.float64),
                            torch.ones(n_pages, dtype=torch.float64), page)
    q = torch.zeros(H, D)
    q[:, 0] = torch.tensor([60.0, -60.0, 500.0, -500.0, 5.0, -5.0, 0.0, 1.0])
    q[4:, 1] = 20.0
    table = torch.arange(n_pages, dtype=torch.int32)[None].contiguous()
    sink = torch.zeros(H)
    pos = torch.arange(n)
    got = call(q.bfloat16(), val, scale, table, sink, n)
    check(got, attn64(q.bfloat16(), val, scale, sink, pos // page, pos % page, D ** -0.5))

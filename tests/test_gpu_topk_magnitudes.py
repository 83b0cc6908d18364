"""The selection at magnitudes far from 1: key rows whose squares leave fp32's range, subnormal
elements and weights, borders that only sums of more than fp32's bits can tell."""
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import indexer_topk, paged_indexer_topk
from tests import _topk as ref

pytestmark = pytest.mark.gpu


def _close_scores(n, H, D, seed):
    """Keys that differ in a few last bits: scores within the tensor core's error of one another."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.rand(1, 3, H, D, generator=g, device="cuda") + 0.5).bfloat16()
    k = (torch.rand(D, generator=g, device="cuda") + 1.0).bfloat16().expand(1, n, D).clone()
    at = torch.randint(0, D, (n,), generator=g, device="cuda")
    k.view(torch.int16)[0, torch.arange(n, device="cuda"), at] += torch.randint(-2, 3, (n,), generator=g, device="cuda", dtype=torch.int16)
    w = torch.rand(1, 3, H, generator=g, device="cuda") + 0.5
    w[0, 1] *= -1
    return q, w, k


def _times(x, e):
    """x 2^e, exact where the type holds it."""
    for part in (e // 2, e - e // 2):
        x = x * torch.tensor(2.0 ** part, dtype=torch.float64, device=x.device).to(x.dtype)
    return x


# log2 of keys, queries and weights.  (Differences of scores here are some 2^-14 of them: above
# 2^-126 (1 + sum |w|), what the choice is defined to.)
SCALES = [(-80, 80, 0), (-100, 60, 20), (-126, 100, 0), (-130, 110, 0), (-60, 0, 0), (0, -100, 30), (60, -100, 60), (0, 0, -90), (90, 10, -128), (80, -60, 0),
          (100, -90, 40)]


@pytest.mark.parametrize("k2,q2,w2", SCALES)
@pytest.mark.parametrize("H,D", [(4, 64), (24, 64), (64, 128)])
def test_borders_closer_than_the_sums(k2, q2, w2, H, D):
    q, w, k = _close_scores(2600, H, D, H + k2)
    q, w, k = _times(q, q2), _times(w, w2), _times(k, k2)
    assert torch.isfinite(q).all() and torch.isfinite(k).all() and w.ne(0).all()
    for topk, block in ((1000, 1), (17, 1), (640, 8)):
        got = indexer_topk(q, w, k, topk, block, check_status=True)
        want = ref.flat(q, w, k, topk, block)
        assert torch.equal(got.long(), want), (topk, block, (got.long() != want).sum(2).tolist())


@pytest.mark.parametrize("k2,q2,w2", SCALES)
def test_ordinary_borders(k2, q2, w2):
    g = torch.Generator(device="cuda").manual_seed(k2 + 200)
    q = _times(torch.randn(1, 10, 16, 128, generator=g, device="cuda").bfloat16(), q2)
    k = _times(torch.randn(1, 2000, 128, generator=g, device="cuda").bfloat16(), k2)
    w = _times(torch.randn(1, 10, 16, generator=g, device="cuda"), w2)
    k[0, 100:400] = 0
    q[0, 3] = 0
    w[0, 4] = 0
    for topk, block in ((500, 1), (512, 64), (1800, 1)):
        assert torch.equal(indexer_topk(q, w, k, topk, block, check_status=True).long(), ref.flat(q, w, k, topk, block)), (topk, block)


@pytest.mark.parametrize("s2,q2,w2", [(-100, 80, 0), (-125, 100, 0), (-20, 0, -80), (0, -100, 10), (100, -90, 0), (0, -80, 60)])
@pytest.mark.parametrize("D,block", [(64, 1), (128, 1), (128, 16)])
def test_paged(s2, q2, w2, D, block):
    n, page, H = 2500, 64, 24
    g = torch.Generator(device="cuda").manual_seed(D + s2)
    code = torch.randint(0x30, 0x40, (1, 1, D), generator=g, device="cuda").expand(-(-n // page), page, D).to(torch.uint8).clone()
    code[:, :, 1] = torch.randint(0, 16, code.shape[:2], generator=g, device="cuda").to(torch.uint8)  # (up to 2^-6 and its neighbours)
    scales = torch.full((code.shape[0],), 2.0 ** s2, device="cuda")
    table = torch.randperm(code.shape[0], generator=g, device="cuda").int()[None]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = _times((torch.rand(2, H, D, generator=g, device="cuda") + 0.5).bfloat16(), q2)
    w = _times(torch.rand(2, H, generator=g, device="cuda") + 0.5, w2)
    w[1] *= -1
    args = (q, w, code.view(torch.float8_e4m3fn), scales, table, i32([n]), i32([0, 0]), i32([n - 2, n - 1]))
    for topk in (5 * block, 60 * block):
        got = paged_indexer_topk(*args, topk, block, check_status=True)
        want = ref.paged(q, w, args[2].double(), scales.double(), *args[4:], topk, block)
        assert torch.equal(got.long(), want), (topk, (got.long() != want).sum(1).tolist())


def test_one_row_of_every_size():
    """Rows from subnormal to near the largest number, beside each other, queries small enough."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q = _times(torch.randn(1, 4, 16, 64, generator=g, device="cuda").bfloat16(), -20)
    w = torch.randn(1, 4, 16, generator=g, device="cuda")
    k = torch.randn(1, 1500, 64, generator=g, device="cuda").double()
    k = (k * torch.exp2(torch.randint(-120, 120, (1500,), generator=g, device="cuda").double())[:, None]).bfloat16()
    for topk, block in ((300, 1), (1200, 1), (256, 16)):
        assert torch.equal(indexer_topk(q, w, k, topk, block, check_status=True).long(), ref.flat(q, w, k, topk, block)), (topk, block)

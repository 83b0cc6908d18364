"""Key rows that hold infinities, at every number of heads (the tensor core's tiles are padded with
heads of zeros, and 0 times infinity is no number)."""
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import indexer_topk
from tests import _topk as ref

pytestmark = pytest.mark.gpu


def _inputs(H, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(1, 20, H, D, generator=g, device="cuda").bfloat16()
    w = torch.randn(1, 20, H, generator=g, device="cuda")
    k = torch.randn(1, 700, D, generator=g, device="cuda").bfloat16()
    rows = torch.randperm(600, generator=g, device="cuda")[:60]
    k[0, rows[:30], 7], k[0, rows[30:], D - 1] = math.inf, -math.inf
    return q, w, k


@pytest.mark.parametrize("H", [1, 5, 16, 24, 33, 64, 65, 100, 128])
def test_selection(H):
    q, w, k = _inputs(H, 64 if H & 1 else 128, H)
    w[0, :4] = w[0, :4].abs()
    w[0, 4:8] = -w[0, 4:8].abs()
    for topk, block in ((20, 1), (300, 1), (672, 1), (128, 8), (256, 64)):
        assert torch.equal(indexer_topk(q, w, k, topk, block, check_status=True).long(), ref.flat(q, w, k, topk, block)), (topk, block)

"""Key rows that hold infinities, at every number of heads (the tensor core's tiles are padded with
heads of zeros, and 0 times infinity is no number)."""
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import indexer_scores_bwd, indexer_scores_fwd
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
def test_scores(H):
    q, w, k = _inputs(H, 64 if H & 1 else 128, H)
    idx = torch.arange(700, dtype=torch.int32, device="cuda").expand(1, 20, 700).contiguous()
    got = indexer_scores_fwd(q, w, k, idx, check_status=True)[0].double()
    for t in range(20):
        want = ref.scores(q[0, t], w[0, t], k[0])
        fin = torch.isfinite(want)
        assert torch.equal(got[t].isnan(), want.isnan()) and torch.equal(got[t].isinf(), want.isinf())
        assert torch.equal(got[t][want.isinf()], want[want.isinf()])
        # (D + 16) 2^-24 of a logit's lengths, (H / 4 + 4) 2^-24 of the sum over heads.
        size = (w[0, t].double().abs() * q[0, t].double().norm(dim=1)).sum() * k[0][fin].double().norm(dim=1)
        assert ((got[t][fin] - want[fin]).abs() <= (q.shape[3] + 16 + H / 4 + 4) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("H", [5, 24, 100])
def test_gradient_of_the_weights(H):
    """dweights of a gradient on one infinite logit: infinite or NaN for that head alone as the
    formula has it."""
    q, w, k = _inputs(H, 128, H)
    idx = k[0, :, 7].isinf().nonzero()[:1].int().expand(1, 20, 1).contiguous()
    g = torch.ones(1, 20, 1, device="cuda")
    dw = indexer_scores_bwd(q, w, k, idx, g, check_status=True)[1]
    x = torch.einsum("shd,d->sh", q[0].double(), k[0, idx[0, 0, 0]].double())
    want = torch.where(x.isnan(), x, x.clamp(min=0))
    assert torch.equal(dw[0].isnan(), want.isnan()) and torch.equal(dw[0].isinf(), want.isinf())

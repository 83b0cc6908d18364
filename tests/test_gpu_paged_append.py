"""The cache's write where a page's scale grows again and again: what the codes stand for against
the rows themselves, and calls of the attention without positions."""
import pytest
import torch

from bwd_sparse_mqa_gb300 import paged_kv_append, sparse_mqa_paged_fwd
from tests import _paged as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 512])
@pytest.mark.parametrize("page,step", [(16, 1.5), (32, 0.7), (128, 0.1)])
def test_append_token_by_token_under_growing_scales(D, page, step):
    """Rows of a wide range of magnitudes, the largest last. At once, a value is off by its
    rounding, half a step of e4m3: 2^-4 of it, or 2^-10 s where its code is subnormal. One row at
    a time, each growth of the scale to s rounds the codes that become subnormal once more, by
    2^-10 s; the scales at least double from one growth to the next, so that all of them
    together come to less than 2^-9 of the last one."""
    g = torch.Generator().manual_seed(D + page)
    new = torch.randn(page, D, generator=g) * torch.exp2(step * torch.arange(page)[:, None] +
                                                         12 * torch.rand(page, D, generator=g) - 12)
    new = new.bfloat16()
    slot = torch.arange(page, dtype=torch.int32, device="cuda")
    cache = [torch.zeros(1, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scale = [torch.ones(1, device="cuda") for _ in range(2)]
    paged_kv_append(new.cuda(), slot, cache[0], scale[0])
    val, sc = torch.zeros(1, page, D, dtype=torch.float64), torch.ones(1, dtype=torch.float64)
    growths, had = 0, 0.0
    for i in range(page):
        paged_kv_append(new[i:i + 1].cuda(), slot[i:i + 1], cache[1], scale[1])
        val, sc = ref.append(new[i:i + 1], [i], val, sc, page)
        growths, had = growths + (float(sc) > had), float(sc)
    assert growths > 5 and torch.equal(ref.codes(cache[1]), val) and torch.equal(scale[1].cpu().double(), sc)
    assert torch.equal(scale[0], scale[1])
    x, s = new.double(), float(sc)
    for c, twice in ((cache[0], 0.0), (cache[1], 2.0 ** -9 * s)):
        off = (ref.codes(c)[0] * s - x).abs() - torch.maximum(2.0 ** -4 * x.abs(), torch.full_like(x, 2.0 ** -10 * s))
        assert float(off.max()) <= twice
    assert not torch.equal(cache[0].view(torch.uint8), cache[1].view(torch.uint8))  # (they do differ)


@pytest.mark.parametrize("D", [64, 512])
def test_attn_with_a_list_needs_no_positions(D):
    g = torch.Generator().manual_seed(D)
    cache, scale = ref.fill_cache(20, 16, D, 2)
    table, _ = ref.deal([200, 100], 16, 13, 20, 3)
    req = torch.tensor([0, 1, -1, 0], dtype=torch.int32)
    q, sink = torch.randn(4, 33, D, generator=g).bfloat16(), torch.randn(33, generator=g)
    idx = torch.randint(-5, 210, (4, 150), generator=g).int()
    seq = torch.tensor([200, 100], dtype=torch.int32)
    args = [x.cuda() for x in (q, cache, scale, sink, table, seq, req)]
    got = sparse_mqa_paged_fwd(*args, topk_idxs=idx.cuda())
    same = sparse_mqa_paged_fwd(*args, torch.zeros(4, dtype=torch.int32, device="cuda"), idx.cuda())
    assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])
    ref.check_attn(got, ref.attn(q, ref.codes(cache), scale.double(), sink, table, seq, req, idx=idx))

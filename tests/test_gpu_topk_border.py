"""The selection where nearly every token's border is scored a second time: many calls in a row, each
compared, by the kernels of 256 and of 1024 threads, over contiguous and paged keys."""
import pytest
import torch

from bwd_sparse_mqa_gb300 import indexer_topk, paged_indexer_topk
from bwd_sparse_mqa_gb300.api import device_status
from tests import _topk as ref

pytestmark = pytest.mark.gpu


def _keys(n, D, seed):
    """Rows in groups of eight that differ in the last bits of one small element: 2^-8 of 2^-6 of one
    of D products, far less than a score's error bound (some 2^-16 of the product of the lengths)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(n // 8, D, generator=g, device="cuda").bfloat16().repeat_interleave(8, 0)
    k[:, 3] = torch.tensor(2.0 ** -6, device="cuda") * (1 + torch.arange(8, device="cuda").repeat(n // 8) / 128)
    return k[torch.randperm(n, generator=g, device="cuda")].contiguous(), g


@pytest.mark.parametrize("S,S_kv,topk", [(300, 4096, 500), (150, 6000, 501)])  # (256 threads; 1024: up to 152 tokens of longer rows)
def test_every_call_is_the_same(S, S_kv, topk):
    k, g = _keys(S_kv, 128, S)
    q = torch.randn(1, S, 64, 128, generator=g, device="cuda").bfloat16()
    w = torch.randn(1, S, 64, generator=g, device="cuda") * 0.01
    first = indexer_topk(q, w, k[None], topk, check_status=True)
    for t in (0, 1, S // 2, S - 1):
        want = ref.choose(ref.scores(q[0, t], w[0, t], k[:S_kv - S + t + 1]), topk)
        assert torch.equal(first[0, t].long(), want), t
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(1000):
        wrong += (indexer_topk(q, w, k[None], topk) != first).sum()
    assert int(wrong) == 0 and device_status() == 0


@pytest.mark.parametrize("R,n,topk", [(200, 2048, 300), (100, 6000, 301)])
def test_every_paged_call_is_the_same(R, n, topk):
    k, g = _keys(n, 128, R)
    page = 64
    cache = torch.zeros(-(-n // page), page, 128, device="cuda").to(torch.float8_e4m3fn)
    cache.view(-1, 128)[:n].copy_(k.float().to(torch.float8_e4m3fn))
    code = cache.view(torch.uint8).view(-1, 128)[:n]
    code[:, 3] = torch.arange(n, device="cuda", dtype=torch.int64).remainder(8).to(torch.uint8) + 8  # (2^-6 and up)
    scales = torch.ones(cache.shape[0], device="cuda")
    table = torch.arange(cache.shape[0], dtype=torch.int32, device="cuda").expand(R, -1).contiguous()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    seq, req = i32([n - r for r in range(R)]), i32(list(range(R)))
    q = torch.randn(R, 64, 128, generator=g, device="cuda").bfloat16()
    w = torch.randn(R, 64, generator=g, device="cuda") * 0.01
    args = (q, w, cache, scales, table, seq, req, None, topk)
    first = paged_indexer_topk(*args, check_status=True)
    val = cache.view(torch.uint8).view(torch.float8_e4m3fn).double().view(-1, 128)
    for t in (0, 1, R - 1):
        assert torch.equal(first[t].long(), ref.choose(ref.scores(q[t], w[t], val[:n - t]), topk)), t
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(1000):
        wrong += (paged_indexer_topk(*args) != first).sum()
    assert int(wrong) == 0 and device_status() == 0


def _close_scores(n, H, D, seed):
    """Keys that differ in a few last bits and scores of one sign: every block's best row is scored again."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.rand(1, 3, H, D, generator=g, device="cuda") + 0.5).bfloat16()
    k = (torch.rand(D, generator=g, device="cuda") + 1.0).bfloat16().expand(1, n, D).clone()
    at = torch.randint(0, D, (n,), generator=g, device="cuda")
    k.view(torch.int16)[0, torch.arange(n, device="cuda"), at] += torch.randint(-2, 3, (n,), generator=g, device="cuda", dtype=torch.int16)
    w = torch.rand(1, 3, H, generator=g, device="cuda") + 0.5
    return q, w, k, g


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("H,D", [(1, 64), (16, 64), (24, 128), (64, 128)])
@pytest.mark.parametrize("n,block", [(2600, 8), (9000, 2), (9000, 64)])
def test_rows_that_are_no_numbers_in_blocks_scored_again(bad, H, D, n, block):
    """A row of a NaN logit ranks last, one of an infinite logit where its weights' signs put it; the
    rest of its block decides with the numbers that it has."""
    q, w, k, g = _close_scores(n, H, D, n + H)
    rows = torch.randperm(n, generator=g, device="cuda")[:n // 20]
    k[0, rows, torch.randint(0, D, (len(rows),), generator=g, device="cuda")] = bad
    w[0, 1] *= -1
    w[0, 2, ::2] *= -1
    for topk in (4 * block, 20 * block, 40 * block):
        got = indexer_topk(q, w, k, topk, block, check_status=True)
        want = ref.flat(q, w, k, topk, block)
        assert torch.equal(got.long(), want), (topk, (got.long() != want).sum(2).tolist())


@pytest.mark.parametrize("D,block", [(64, 8), (128, 16), (128, 64)])
def test_nan_codes_in_blocks_scored_again(D, block):
    n, page, H = 3000, 64, 16
    g = torch.Generator(device="cuda").manual_seed(D + block)
    code = torch.randint(0x38, 0x3a, (-(-n // page), page, D), generator=g, device="cuda").to(torch.uint8)  # (1 and 1.125)
    code[:, :, 1:] = code[0, 0, 1:]
    code[:, :, 0] = torch.randint(8, 16, code.shape[:2], generator=g, device="cuda").to(torch.uint8)  # (2^-6 and up)
    code.view(-1, D)[torch.randperm(n, generator=g, device="cuda")[:n // 20], 5] = 0x7f
    cache, scales = code.view(torch.float8_e4m3fn), torch.full((code.shape[0],), 0.5, device="cuda")
    table = torch.randperm(code.shape[0], generator=g, device="cuda").int()[None]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = (torch.rand(2, H, D, generator=g, device="cuda") + 0.5).bfloat16()
    w = torch.rand(2, H, generator=g, device="cuda") + 0.5
    w[1] *= -1
    args = (q, w, cache, scales, table, i32([n]), i32([0, 0]), i32([n - 2, n - 1]))
    for blocks in (3, 9):
        got = paged_indexer_topk(*args, blocks * block, block, check_status=True)
        want = ref.paged(q, w, cache.double(), scales.double(), *args[4:], blocks * block, block)
        assert torch.equal(got.long(), want), (blocks, (got.long() != want).sum(1).tolist())

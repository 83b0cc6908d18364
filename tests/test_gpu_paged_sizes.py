"""The paged-cache operators at sizes where 32-bit sums and roundings end."""
import pytest
import torch

from bwd_sparse_mqa_gb300 import paged_plan, paged_release

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _room(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


@pytest.mark.parametrize("inplace", [False, True])
def test_plan_of_more_pages_than_an_int(inplace):
    """All requests together need more than 2^31 pages: the stack's few go to the first request,
    every other entry is -1, and the count ends at the most negative one it can."""
    _room(32)
    R, W, page = 16384, 131073, 16
    table = torch.full((R, W), 7, dtype=torch.int32, device="cuda")
    got = paged_plan(torch.zeros(R, dtype=torch.int32, device="cuda"),
                     torch.full((R,), W * page, dtype=torch.int32, device="cuda"), table, _i32([11, 12, 13, 14, 15]),
                     _i32([5]), page, 40, 100, inplace=inplace)
    assert got.block_table[0, :6].tolist() == [15, 14, 13, 12, 11, -1]
    got.block_table[0, :5] = -1
    assert all(int(part.max()) == int(part.min()) == -1 for part in got.block_table.split(1024))
    assert int(got.free_count) == 5 - (2 ** 31 - 1)
    assert got.token_req.tolist() == [0] * 40 and got.slot_mapping.tolist() == [15 * 16 + i for i in range(16)] + \
        [14 * 16 + i for i in range(16)] + [13 * 16 + i for i in range(8)]


def test_release_onto_a_full_stack_as_long_as_an_int():
    """A stack of 2^31 - 1 entries with room for three: the rest is dropped, nothing is written
    outside of the stack, and the count ends at its length."""
    _room(24)
    pool = 2 ** 31 - 1
    free = torch.full((pool,), -5, dtype=torch.int32, device="cuda")
    table = torch.arange(100, dtype=torch.int32, device="cuda").view(2, 50).contiguous()
    count, gone = _i32([pool - 3]), torch.tensor([True, True], device="cuda")
    paged_release(table, gone, free, count, 100)
    assert int(count) == pool and free[-3:].tolist() == [0, 1, 2]
    assert int(free[:-3].max()) == int(free[:-3].min()) == -5 and int(table.max()) == -1


@pytest.mark.parametrize("inplace", [False, True])
def test_plan_of_as_many_token_rows_as_an_int(inplace):
    """max_tokens up to 2^31 - 1: every row behind the tokens is -1, and nothing else is written."""
    _room(64)
    N = 2 ** 31 - 1
    plan = paged_plan(_i32([3, 0]), _i32([2, 1]), _i32([[4], [-1]]), _i32([6]), _i32([1]), 16, N, 9, inplace=inplace)
    assert plan.token_req[:4].tolist() == [0, 0, 1, -1] and plan.positions[:4].tolist() == [3, 4, 0, -1]
    assert plan.slot_mapping[:4].tolist() == [67, 68, 96, -1]
    for t in (plan.token_req, plan.positions, plan.slot_mapping):
        assert t.numel() == N and int(t[3:].max()) == int(t[3:].min()) == -1
    assert plan.seq_lens.tolist() == [5, 1] and plan.cu_query.tolist() == [0, 2, 3]

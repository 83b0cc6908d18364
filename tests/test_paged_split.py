"""When the attention splits tokens between ranges (it asks for a workspace then): the rule on
the host, checked without a GPU."""
import pytest

from bwd_sparse_mqa_gb300 import _lib


def _split(T, H, D, topk):
    return _lib.load().smqa_paged_fwd_workspace_bytes(_lib.PagedShape(T, T, H, D, topk, 64, 2048, 4096)) > 0


@pytest.mark.parametrize("D", [64, 512])
@pytest.mark.parametrize("H", [16, 64, 65, 128])
@pytest.mark.parametrize("T", [1, 2, 4, 8])
def test_few_tokens_with_long_lists_are_split(T, H, D):
    """Most SMs would stay idle: a lone token's 8 or 12 blocks one after another took 22.8 and
    29.5 us, more than 16 blocks split (17.4)."""
    assert all(_split(T, H, D, topk) for topk in (1024, 1536, 2048, 4096, 8192))


@pytest.mark.parametrize("D", [64, 512])
@pytest.mark.parametrize("T", [1, 8, 32, 76, 152, 1000])
def test_short_lists_are_not(T, D):
    assert not any(_split(T, 128, D, topk) for topk in (1, 32, 128, 256))


@pytest.mark.parametrize("D", [64, 512])
@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 20, 33, 60])
def test_longer_lists_stay_split(T, H, D):
    """More blocks per token only ever speak for splitting."""
    at = [_split(T, H, D, 128 * nb) for nb in range(1, 200)]
    first = at.index(True)
    assert all(at[first:])

"""Sizes that the selections refuse (host checks, without a GPU): their kernels' loops over a list's
entries and over the positions that a token sees step by up to 1024 threads, in 32 bits."""
import ctypes

import pytest

from bwd_sparse_mqa_gb300 import _lib

LIM = 2 ** 31 - 2048
P = ctypes.c_void_p(0x10000)


def _flat(S_kv, topk, block=1):
    """(workspace bytes, status) of a call that no GPU runs: its workspace is always too small."""
    lib, shp = _lib.load(), _lib.Shape(1, 1, S_kv, 16, 64, topk)
    st = lib.smqa_indexer_topk(P, P, P, shp, block, 0, 0, P, P, 0, None)
    return lib.smqa_indexer_topk_workspace_bytes(shp, block), st, lib.smqa_last_error()


def _paged(positions, topk, page=16, block=1):
    lib, shp = _lib.load(), _lib.PagedShape(1, 1, 16, 64, topk, page, positions // page, 10)
    st = lib.smqa_paged_indexer_topk(*[P] * 8, shp, block, 0, P, P, 0, 0, None)
    return lib.smqa_paged_indexer_topk_workspace_bytes(shp, block), st, lib.smqa_last_error()


@pytest.mark.parametrize("topk,block", [(LIM + 1, 1), (LIM + 1024, 1), (2 ** 31 - 256, 1), (2 ** 31 - 1, 1), (LIM + 128, 128), (2 ** 31 - 128, 128)])
@pytest.mark.parametrize("call", [_flat, _paged])
def test_lists_too_long(call, topk, block):
    need, st, why = call(4096, topk, block=block)
    assert need == 0 and st == _lib.SMQA_ERR_UNSUPPORTED and b"topk" in why


@pytest.mark.parametrize("n", [LIM + 1, 2 ** 31 - 512, 2 ** 31 - 256])
def test_too_many_positions(n):
    need, st, why = _flat(n, 64)
    assert need == 0 and st == _lib.SMQA_ERR_UNSUPPORTED and b"S_kv" in why
    for page in (16, 128):
        need, st, why = _paged(-(-n // page) * page, 64, page)
        assert need == 0 and st == _lib.SMQA_ERR_UNSUPPORTED and b"max_pages" in why


@pytest.mark.parametrize("call", [_flat, _paged])
def test_the_largest_are_taken(call):
    for n, topk, block in ((LIM, 64, 1), (4096, LIM, 1), (4096, LIM, 128), (LIM, LIM, 128)):
        need, st, why = call(n, topk, block=block)
        assert need > 0 and st == _lib.SMQA_ERR_UNSUPPORTED and b"workspace too small" in why, (n, topk, block)

"""Sizes the attention over the paged cache refuses (host checks, without a GPU): the number of a
token's blocks of 128 slots is rounded up in 32 bits."""
import ctypes

import pytest

from bwd_sparse_mqa_gb300 import _lib

LIM = 2 ** 31 - 128


@pytest.mark.parametrize("topk", [LIM + 1, LIM + 100, 2 ** 31 - 1])
def test_lists_too_long_are_refused(topk):
    p, lib = ctypes.c_void_p(0x10000), _lib.load()
    shp = _lib.PagedShape(1, 1, 1, 64, topk, 16, 4, 10)
    assert lib.smqa_paged_fwd(*[p] * 9, shp, 0.0, p, p, p, 1 << 50, 0, None) == _lib.SMQA_ERR_UNSUPPORTED
    assert b"2^31" in lib.smqa_last_error() and lib.smqa_paged_fwd_workspace_bytes(shp) == 0


@pytest.mark.parametrize("page", [16, 32, 64])
def test_tables_too_wide_are_refused(page):
    p, lib = ctypes.c_void_p(0x10000), _lib.load()
    shp = _lib.PagedShape(1, 1, 1, 64, 0, page, 2 ** 31 // page - 1, 10)
    assert lib.smqa_paged_fwd(*[p] * 8, None, shp, 0.0, p, p, p, 1 << 50, 0, None) == _lib.SMQA_ERR_UNSUPPORTED
    assert lib.smqa_paged_fwd_workspace_bytes(shp) == 0


def test_the_largest_are_taken():
    lib = _lib.load()
    assert lib.smqa_paged_fwd_workspace_bytes(_lib.PagedShape(1, 1, 1, 64, LIM, 16, 4, 10)) > 0
    assert lib.smqa_paged_fwd_workspace_bytes(_lib.PagedShape(1, 1, 1, 64, 0, 16, LIM // 16, 10)) > 0
    assert lib.smqa_paged_fwd_workspace_bytes(_lib.PagedShape(1, 1, 1, 64, 0, 128, LIM // 128, 10)) > 0

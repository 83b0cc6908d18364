"""Lists that the attention, the indexer's backward and its scores refuse (host checks, without a
GPU): their kernels' loops over a token's slots step by up to 384 threads, in 32 bits."""
import ctypes

import pytest

from bwd_sparse_mqa_gb300 import _lib

LIM = 2 ** 31 - 2048
P = ctypes.c_void_p(0x10000)


def _calls(topk):
    """Statuses of calls that launch nothing whatever topk is: each lacks a pointer."""
    lib = _lib.load()
    a, i = _lib.Shape(1, 1, 100, 16, 64, topk), _lib.Shape(1, 1, 100, 16, 64, topk)
    yield lib.smqa_fwd(P, P, P, P, a, 0.1, P, None, None, 0, 0, None)
    yield lib.smqa_bwd(P, P, P, P, P, P, P, a, 0.1, P, P, None, None, 0, 0, None)
    yield lib.smqa_indexer_bwd(P, P, P, P, P, i, None, None)
    yield lib.smqa_batched_indexer_bwd(P, P, P, P, P, i, None, None)
    yield lib.smqa_indexer_scores(P, P, P, P, i, None, None)
    yield lib.smqa_indexer_scores_bwd(P, P, P, P, P, i, P, P, None, P, 1 << 40, 0, None)


@pytest.mark.parametrize("topk", [LIM + 1, 2 ** 31 - 384, 2 ** 31 - 128, 2 ** 31 - 1])
def test_lists_too_long(topk):
    assert list(_calls(topk)) == [_lib.SMQA_ERR_UNSUPPORTED] * 6
    assert b"topk" in _lib.load().smqa_last_error()
    assert _lib.load().smqa_bwd_workspace_bytes(_lib.Shape(1, 1, 100, 16, 64, topk), 0) == 0


def test_the_longest_are_taken():
    assert list(_calls(LIM)) == [_lib.SMQA_ERR_INVALID_ARG] * 6  # (past the sizes: the pointer)
    assert _lib.load().smqa_bwd_workspace_bytes(_lib.Shape(1, 1, 100, 16, 64, LIM), 0) > 0

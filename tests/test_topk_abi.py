"""Refusals of the selection's and the scores' C entries (host checks: they run without a GPU), and
the plain choice the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import _lib, indexer_scores_fwd, indexer_topk, paged_indexer_topk
from tests import _topk as ref

INVALID, UNSUPPORTED, OK = _lib.SMQA_ERR_INVALID_ARG, _lib.SMQA_ERR_UNSUPPORTED, _lib.SMQA_OK


def _p(addr=0x10000):
    return ctypes.c_void_p(addr)


def test_topk_refusals():
    lib = _lib.load()

    def call(q=_p(), w=_p(), k=_p(), B=1, S=4, S_kv=100, H=16, D=64, topk=8, block=1, recent=0, out=_p(), ws=_p(), n=1 << 40):
        shp = _lib.Shape(B, S, S_kv, H, D, topk)
        return lib.smqa_indexer_topk(q, w, k, shp, block, recent, 0, out, ws, n, None)
    for bad in ({"B": 0}, {"S": 0}, {"S_kv": 0}, {"H": 0}, {"D": 0}, {"topk": 0}, {"block": 0}, {"recent": -1}, {"recent": 9}):
        assert call(**bad) == INVALID, bad
    for bad in ({"H": 129}, {"D": 512}, {"block": 3}, {"block": 256, "topk": 256}, {"block": 16}, {"S_kv": 2 ** 31 - 1}, {"B": 2 ** 20, "S_kv": 2 ** 11},
                {"B": 2 ** 20, "S": 2 ** 11}):
        assert call(**bad) == UNSUPPORTED, bad
    for name in ("q", "w", "k", "out", "ws"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: _p(0x10002)}) == INVALID, name
    for name in ("q", "k", "ws"):
        assert call(**{name: _p(0x10008)}) == INVALID, name
    need = lib.smqa_indexer_topk_workspace_bytes(_lib.Shape(1, 4, 100, 16, 64, 8), 1)
    assert need >= 4 * 100 * 4 and call(n=need - 1) == UNSUPPORTED and b"workspace too small" in lib.smqa_last_error()
    assert lib.smqa_indexer_topk_workspace_bytes(_lib.Shape(1, 4, 100, 16, 32, 8), 1) == 0
    assert lib.smqa_indexer_topk_workspace_bytes(_lib.Shape(1, 4, 100, 16, 64, 8), 3) == 0
    # Long rows and many tokens: a chunk of scores, not all of them.
    assert lib.smqa_indexer_topk_workspace_bytes(_lib.Shape(1, 2 ** 20, 2 ** 20, 64, 128, 2048), 1) < 1 << 30


def test_paged_topk_refusals():
    lib = _lib.load()

    def call(at=None, ptr=None, T=2, R=2, H=16, D=64, topk=8, page=16, W=4, n=10, block=1, recent=0, out=_p(), ws=_p(), nb=1 << 40, flags=0):
        a = [_p()] * 8
        if at is not None:
            a[at] = ptr
        return lib.smqa_paged_indexer_topk(*a, _lib.PagedShape(T, R, H, D, topk, page, W, n), block, recent, out, ws, nb, flags, None)
    for at in range(7):
        assert call(at) == INVALID and call(at, _p(0x10002)) == INVALID
    assert call(7, _p(0x10002)) == INVALID                # (positions may be NULL)
    assert call(0, _p(0x10008)) == INVALID and call(2, _p(0x10008)) == INVALID
    assert call(out=None) == INVALID and call(ws=None) == INVALID and call(ws=_p(0x10010)) == INVALID and call(flags=1) == INVALID
    for bad in ({"T": -1}, {"R": 0}, {"H": 0}, {"D": 0}, {"topk": 0}, {"page": 0}, {"W": 0}, {"n": 0}, {"recent": 9}):
        assert call(**bad) == INVALID, bad
    for bad in ({"H": 129}, {"D": 512}, {"page": 8}, {"page": 24}, {"n": 1 << 28}, {"W": 1 << 28}, {"block": 5}, {"block": 16}):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(T=0) == OK
    need = lib.smqa_paged_indexer_topk_workspace_bytes(_lib.PagedShape(2, 2, 16, 64, 8, 16, 4, 10), 1)
    assert need > 0 and call(nb=need - 1) == UNSUPPORTED


def test_scores_refusals():
    lib = _lib.load()

    def fwd(at=None, ptr=None, B=1, S=4, S_kv=100, H=16, D=64, topk=8):
        a = [_p()] * 5
        if at is not None:
            a[at] = ptr
        return lib.smqa_indexer_scores(*a[:4], _lib.Shape(B, S, S_kv, H, D, topk), a[4], None)

    def bwd(at=None, ptr=None, B=1, S=4, S_kv=100, H=16, D=64, topk=8, n=1 << 40, flags=0):
        a = [_p()] * 9
        if at is not None:
            a[at] = ptr
        return lib.smqa_indexer_scores_bwd(*a[:5], _lib.Shape(B, S, S_kv, H, D, topk), *a[5:], n, flags, None)
    for at in range(5):
        assert fwd(at) == INVALID and fwd(at, _p(0x10002)) == INVALID
    for at in range(9):
        assert bwd(at) == INVALID and bwd(at, _p(0x10002)) == INVALID
    for f in (fwd, bwd):
        for bad in ({"B": 0}, {"S": 0}, {"S_kv": 0}, {"H": 0}, {"D": 0}, {"topk": 0}):
            assert f(**bad) == INVALID, bad
        for bad in ({"H": 129}, {"D": 512}, {"B": 2 ** 20, "S": 2 ** 10}, {"B": 2 ** 20, "S_kv": 2 ** 11}, {"topk": 2 ** 31 - 1}):
            assert f(**bad) == UNSUPPORTED, bad
    assert bwd(flags=2) == INVALID
    shp = _lib.Shape(1, 4, 100, 16, 64, 8)
    assert lib.smqa_indexer_scores_bwd_workspace_bytes(shp, 0) == 100 * 64 * 4 and bwd(n=100 * 64 * 4 - 1) == UNSUPPORTED
    assert lib.smqa_indexer_scores_bwd_workspace_bytes(shp, _lib.FLAG_RETURN_DKV_FP32) == 0


def test_python_refuses_cpu_tensors():
    q, w, k = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 4), torch.zeros(1, 9, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        indexer_topk(q, w, k, 4)
    with pytest.raises(ValueError, match="CUDA"):
        indexer_scores_fwd(q, w, k, torch.zeros(1, 2, 3, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        paged_indexer_topk(q[0], w[0], torch.zeros(3, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(3), i[:, None], i, i, i, 4)


def test_plain_choice():
    s = torch.tensor([1.0, 3.0, 3.0, math.nan, -1.0, 3.0, math.inf, -math.inf, 0.0, -0.0], dtype=torch.float64)
    assert ref.choose(s, 3).tolist() == [1, 2, 6]
    assert ref.choose(s, 4).tolist() == [1, 2, 5, 6]
    assert ref.choose(s, 6).tolist() == [0, 1, 2, 5, 6, 8]
    assert ref.choose(s, 9).tolist() == [0, 1, 2, 4, 5, 6, 7, 8, 9]
    assert ref.choose(s, 12).tolist() == list(range(10)) + [-1, -1]
    assert ref.choose(s, 4, recent=2).tolist() == [1, 6, 8, 9]
    assert ref.choose(s, 4, block=4).tolist() == [4, 5, 6, 7]
    assert ref.choose(s, 8, block=4, recent=1).tolist() == [4, 5, 6, 7, 8, 9, -1, -1]
    there = torch.ones(10, dtype=torch.bool)
    there[[1, 6]] = False
    assert ref.choose(s, 3, there=there).tolist() == [0, 2, 5]
    assert ref.choose(s, 4, block=2, there=there).tolist() == [2, 3, 4, 5]

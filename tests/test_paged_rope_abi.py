"""Refusals of the rotated paged append (host checks: they run without a GPU)."""
import ctypes

import pytest
import torch

from bwd_sparse_mqa_gb300 import _lib, paged_kv_append

INVALID, UNSUPPORTED, OK = _lib.SMQA_ERR_INVALID_ARG, _lib.SMQA_ERR_UNSUPPORTED, _lib.SMQA_OK


def _p(addr=0x10000):
    return ctypes.c_void_p(addr)


def test_refusals():
    fn = _lib.load().smqa_paged_append_rope

    def call(new=_p(), slots=_p(), pos=_p(), cs=_p(), T=1, D=128, page=16, n=9, rows=100, dim=64, off=0, inter=0,
             cache=_p(), scales=_p()):
        return fn(new, slots, pos, cs, T, D, page, n, rows, dim, off, inter, cache, scales, None)
    for bad in ({"T": -1}, {"D": 0}, {"page": 0}, {"n": 0}, {"rows": -1}, {"dim": -16}, {"off": -8}):
        assert call(**bad) == INVALID, bad
    for bad in ({"D": 256}, {"D": 96}, {"page": 24}, {"page": 128, "n": 1 << 24}, {"dim": 8}, {"dim": 144},
                {"dim": 40}, {"off": 4}, {"off": 72}, {"off": 2 ** 31 - 8}):
        assert call(**bad) == UNSUPPORTED, bad
    for name in ("new", "slots", "pos", "cs", "cache", "scales"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: _p(0x10002)}) == INVALID, name
    for name in ("new", "cs", "cache"):
        assert call(**{name: _p(0x10008)}) == INVALID, name
    assert call(T=0, new=None, slots=None, pos=None, cs=None, cache=None, scales=None) == OK


def test_python_refuses_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(3, 16, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA"):
        paged_kv_append(torch.zeros(2, 128, dtype=torch.bfloat16), i, cache, torch.ones(3), positions=i,
                        cos_sin=torch.ones(4, 64))

"""Refusals of the paged-cache entry points (host checks: they run without a
GPU), and the plain forms the GPU tests compare with, checked on the CPU."""
import ctypes
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import _lib, paged_kv_append, paged_plan, paged_release, sparse_mqa_paged_fwd
from tests import _paged as ref

INVALID, UNSUPPORTED = _lib.SMQA_ERR_INVALID_ARG, _lib.SMQA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _p(addr=0x10000):
    return ctypes.c_void_p(addr)


def test_plan_refusals(lib):
    def call(ptr=None, at=None, R=4, W=4, page=16, n_pages=100, pool=10, N=8, out=None):
        a = [_p(0x10000 + 0x1000 * i) for i in range(5)]
        b = [_p(0x20000 + 0x1000 * i) for i in range(7)]
        if at is not None:
            (a if at < 5 else b)[at if at < 5 else at - 5] = ptr
        if out:
            for i, j in out:
                b[i] = a[j]
        return lib.smqa_paged_plan(*a, R, W, page, n_pages, pool, N, *b, None)
    for at in range(12):
        assert call(None, at) == INVALID
        assert call(_p(0x10002), at) == INVALID
    for bad in ({"R": 0}, {"W": 0}, {"page": 0}, {"n_pages": 0}, {"pool": -1}, {"N": -1}):
        assert call(**bad) == INVALID
    for bad in ({"R": 16385}, {"page": 48}, {"page": 256}, {"n_pages": 1 << 27}, {"W": 1 << 27}):
        assert call(**bad) == UNSUPPORTED
    assert call(out=[(2, 0)]) == INVALID                  # seq_lens over context_lens, count not in place
    assert b"seq_lens" in lib.smqa_last_error()


def test_release_refusals(lib):
    p = _p()
    assert lib.smqa_paged_release(None, p, p, 4, 4, 9, p, p, 9, None) == INVALID
    assert lib.smqa_paged_release(p, p, p, 4, 4, 9, None, p, 9, None) == INVALID
    assert lib.smqa_paged_release(p, _p(0x10001), p, 4, 4, 9, p, p, 9, None) == INVALID
    assert lib.smqa_paged_release(p, p, p, 0, 4, 9, p, p, 9, None) == INVALID
    assert lib.smqa_paged_release(p, p, p, 4, 4, 9, p, p, 0, None) == INVALID


def test_append_refusals(lib):
    p = _p()
    call = lib.smqa_paged_append
    assert call(p, p, -1, 64, 16, 9, p, p, None) == INVALID
    assert call(p, p, 1, 128, 16, 9, p, p, None) == UNSUPPORTED
    assert call(p, p, 1, 64, 24, 9, p, p, None) == UNSUPPORTED
    assert call(p, p, 1, 64, 128, 1 << 24, p, p, None) == UNSUPPORTED
    assert call(_p(0x10008), p, 1, 64, 16, 9, p, p, None) == INVALID
    assert call(p, p, 1, 64, 16, 9, _p(0x10004), p, None) == INVALID
    for i in range(4):
        a = [p, p, p, p]
        a[i] = None
        assert call(a[0], a[1], 1, 64, 16, 9, a[2], a[3], None) == INVALID
    assert call(None, None, 0, 64, 16, 9, None, None, None) == _lib.SMQA_OK   # no rows: nothing to do


def _shape(T=2, R=2, H=16, D=64, topk=8, page=16, W=4, n=10):
    return _lib.PagedShape(T, R, H, D, topk, page, W, n)


def test_fwd_refusals(lib):
    p = _p()

    def call(shp=None, at=None, ptr=None, o=p, lse=p, ws=p, nbytes=1 << 40, flags=0, idx=p, pos=p):
        a = [p] * 7 + [pos, idx]
        if at is not None:
            a[at] = ptr
        return lib.smqa_paged_fwd(*a, shp or _shape(), 0.0, o, lse, ws, nbytes, flags, None)
    for at in range(7):
        assert call(at=at) == INVALID
        assert call(at=at, ptr=_p(0x10002)) == INVALID
    assert call(at=0, ptr=_p(0x10008)) == INVALID
    assert call(o=None) == INVALID and call(lse=None) == INVALID and call(o=_p(0x10008)) == INVALID
    assert call(idx=None) == INVALID                      # topk > 0 without a list
    assert call(_shape(topk=0), pos=None) == INVALID      # no list and no positions
    assert call(ws=_p(0x10010)) == INVALID
    assert call(flags=1) == INVALID and call(flags=32) == INVALID
    for bad in ({"T": -1}, {"R": 0}, {"H": 0}, {"topk": -1}, {"W": 0}, {"n": 0}, {"page": 0}):
        assert call(_shape(**bad)) == INVALID
    for bad in ({"H": 129}, {"D": 128}, {"page": 8}, {"n": 1 << 28}, {"T": 1 << 28}, {"W": 1 << 28},
                {"T": 1 << 12, "topk": 1 << 20}):
        assert call(_shape(**bad)) == UNSUPPORTED
        assert lib.smqa_paged_fwd_workspace_bytes(_shape(**bad)) == 0
    assert call(_shape(T=0)) == _lib.SMQA_OK
    need = lib.smqa_paged_fwd_workspace_bytes(_shape(T=64, D=512, topk=2048))
    if need:
        assert call(_shape(T=64, D=512, topk=2048), nbytes=need - 1) == UNSUPPORTED
        assert b"workspace too small" in lib.smqa_last_error()
        assert call(_shape(T=64, D=512, topk=2048), ws=None) == INVALID


def test_python_refuses_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(3, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA"):
        paged_plan(i, i, i[:, None].contiguous(), i, i[:1], 16, 4, 3)
    with pytest.raises(ValueError, match="CUDA"):
        paged_release(i[:, None].contiguous(), i.bool(), i, i[:1], 3)
    with pytest.raises(ValueError, match="CUDA"):
        paged_kv_append(torch.zeros(2, 64, dtype=torch.bfloat16), i, cache, torch.ones(3))
    with pytest.raises(ValueError, match="CUDA"):
        sparse_mqa_paged_fwd(torch.zeros(2, 4, 64, dtype=torch.bfloat16), cache, torch.ones(3), torch.zeros(4),
                             i[:, None].contiguous(), i, i, i)


@pytest.mark.gpu
def test_python_refuses_what_does_not_match():
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    cache = torch.zeros(3, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = torch.ones(3, device="cuda")
    q, sink = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, device="cuda")
    fwd = lambda **k: sparse_mqa_paged_fwd(**{**dict(q=q, kv_cache=cache, kv_scales=sc, attn_sink=sink, block_table=table, seq_lens=i, token_req=i, positions=i), **k})  # noqa: E731,E501
    fwd()
    for bad in ({"q": q[:, :, :32].contiguous()}, {"attn_sink": sink[:3].contiguous()}, {"seq_lens": i[:1]},
                {"token_req": i[:1]}, {"positions": i[:1]}, {"positions": None}, {"kv_scales": sc[:2]},
                {"topk_idxs": table[:1]}, {"topk_idxs": table[:, :0].contiguous()}, {"out": (q, sink[None])},
                {"q": q.transpose(0, 1)}, {"block_table": table.t()}, {"sm_scale": 0.0}, {"sm_scale": math.nan}):
        with pytest.raises(ValueError):
            fwd(**bad)
    for bad in ({"q": q.half()}, {"kv_cache": cache.view(torch.uint8)}, {"token_req": i.long()}, {"attn_sink": sink.half()},
                {"topk_idxs": table.long()}):
        with pytest.raises(TypeError):
            fwd(**bad)
    with pytest.raises(_lib.SMQAError):
        fwd(kv_cache=torch.zeros(3, 24, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn))
    with pytest.raises(ValueError):
        paged_kv_append(q[0], i, cache, sc)
    with pytest.raises(ValueError):
        paged_plan(i, i[:1], table, i, i[:1], 16, 4, 3)
    with pytest.raises(ValueError):
        paged_plan(i, i, table, i, i[:1], 16, -1, 3)
    with pytest.raises(_lib.SMQAError):
        paged_plan(i, i, table, i, i[:1], 17, 4, 3)
    o, lse = sparse_mqa_paged_fwd(q[:0], cache, sc, sink, table, i, i[:0], i[:0])
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    paged_kv_append(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), i[:0], cache, sc)
    assert paged_plan(i, i, table, i, i[:1], 16, 0, 3).token_req.numel() == 0


def test_plain_e4m3_matches_the_type():
    """Every code is a fixed point; ties between neighbours go to the even code."""
    v = torch.arange(256, dtype=torch.uint8)
    v = v[(v & 0x7f) != 0x7f].view(torch.float8_e4m3fn).float().double()
    assert torch.equal(ref.e4m3(v), v)
    x = torch.linspace(-448, 448, 20001, dtype=torch.float64)
    x = torch.cat([x, x * 2.0 ** -12, torch.tensor([2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -6 * 15.5 / 16])])
    assert torch.equal(ref.e4m3(x), x.float().to(torch.float8_e4m3fn).float().double())


def test_plain_attn_matches_softmax():
    """The plain form against torch's float64 softmax on a dense request with the sink as a column."""
    cache, scale = ref.fill_cache(4, 16, 64, 1, spread=1)
    table, _ = ref.deal([50], 16, 4, 4, 1)
    q = torch.randn(2, 3, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    sink = torch.tensor([0.5, -2.0, float("-inf")])
    o, lse, _, _ = ref.attn(q, ref.codes(cache), scale.double(), sink, table, [50], [0, 0], [49, 10])
    rows = (ref.codes(cache) * scale.double()[:, None, None])[table[0].long()].reshape(-1, 64)
    for t, n in ((0, 50), (1, 11)):
        z = torch.cat([q[t].double() @ rows[:n].T / 8.0, sink.double()[:, None]], 1)
        assert torch.allclose(o[t], torch.softmax(z, 1)[:, :-1] @ rows[:n], rtol=1e-12, atol=1e-12)
        assert torch.allclose(lse[t], torch.logsumexp(z, 1) / math.log(2.0), rtol=1e-12)


@pytest.mark.gpu
def test_python_refuses_sizes_beyond_int32():
    """The C ABI's sizes are int32: a larger one is refused, not cut to its low bits."""
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    for page, tokens, pages in ((16 + 2 ** 32, 4, 3), (16, 4 + 2 ** 32, 3), (16, 4, 3 + 2 ** 32), (16, -1, 3)):
        with pytest.raises(ValueError, match="2\\^31"):
            paged_plan(i, i, table, i, i[:1].clone(), page, tokens, pages)
    with pytest.raises(ValueError, match="2\\^31"):
        paged_release(table, i.bool(), i, i[:1].clone(), 3 + 2 ** 32)
    assert table.eq(0).all()

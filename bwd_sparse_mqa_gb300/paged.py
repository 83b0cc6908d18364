"""Serving over an 8-bit paged kv cache: the step's block table and slots made
on the GPU, the quantising write of new rows, and sparse MQA over the cache.

The cache is a pool of pages, ``kv_cache`` [n_pages, page_size, D]
float8_e4m3fn with one fp32 scale per page, ``kv_scales`` [n_pages]; keys =
values and one kv head, as everywhere in this package.  A step of a server is

    plan = paged_plan(context_lens, query_lens, block_table, free_pages, free_count,
                      page_size, max_tokens, n_pages, inplace=True)
    paged_kv_append(kv_new, plan.slot_mapping, kv_cache, kv_scales)
    o, lse = sparse_mqa_paged_fwd(q, kv_cache, kv_scales, attn_sink, plan.block_table,
                                  plan.seq_lens, plan.token_req, plan.positions, topk_idxs)

Every call is asynchronous on the current stream of its tensors' device, reads
nothing back to the host and can be captured in a CUDA graph.  As in api.py,
PyTorch only supplies device memory and the stream; there is no CPU path.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .api import _check_device, _need, _scale


class PagedPlan(NamedTuple):
    """What paged_plan returns (int32 CUDA tensors)."""
    block_table: torch.Tensor   # [R, max_pages]
    free_count: torch.Tensor    # [1]; negative: that many pages were missing
    seq_lens: torch.Tensor      # [R] context + query
    cu_query: torch.Tensor      # [R + 1]
    token_req: torch.Tensor     # [max_tokens], -1 behind the last token
    positions: torch.Tensor     # [max_tokens], -1 behind the last token
    slot_mapping: torch.Tensor  # [max_tokens], -1 where there is no page


# A step of a server makes a handful of these calls between model layers, and a
# call's kernel may take less time than Python needs to check its arguments:
# the checks of a call are one expression, explained tensor by tensor only when
# it fails, and the stream and device are read without building objects.
_LIM = 2 ** 31                                           # (the C ABI takes sizes as int32)
_I32, _BF16, _F32, _E4M3 = torch.int32, torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _explain(why: str, *tensors: tuple) -> None:
    """Raises what is wrong with the (tensor, name, dtype, ndim) given: the
    first that is not a contiguous CUDA tensor of its type and rank, or that
    lies on another device than the first, else ``why``."""
    for t, name, dtype, ndim in tensors:
        _need(t, name, dtype, ndim)
    if len({t.device for t, *_ in tensors}) != 1:
        raise ValueError("all tensors must be on the same device")
    raise ValueError(why)


def _call(fn: str, device: int, f, *args) -> None:
    """f(*args, current stream of ``device``) with that device current."""
    c = torch._C                                         # (looked up here: a torch without CUDA lacks them)
    if c._cuda_getDevice() == device:
        st = f(*args, c._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            st = f(*args, c._cuda_getCurrentRawStream(device))
    if st != _lib.SMQA_OK:
        _lib.check(fn, st)


def paged_plan(context_lens: torch.Tensor, query_lens: torch.Tensor, block_table: torch.Tensor,
               free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int,
               max_tokens: int, n_pages: int, inplace: bool = False) -> PagedPlan:
    """Block table, offsets, positions and cache slots of one step (C ABI
    ``smqa_paged_plan``; one launch).

    context_lens, query_lens [R]: tokens each request has, and adds now.
    block_table [R, max_pages]: the pages it holds.  free_pages [pool] and
    free_count [1]: a stack of free page ids, its top last.  All int32 CUDA
    tensors.  Each new page a request needs is popped from the stack, requests
    in order; once it is empty the entry and its tokens' slots are -1 and
    free_count ends negative by the pages missing.  max_tokens is the length of
    the token outputs; rows behind the last token are -1.  ``inplace`` updates
    block_table and free_count themselves instead of returning new ones.
    """
    try:
        dev = block_table.get_device()
        R, W = block_table.shape
        ok = (dev >= 0 and context_lens.dtype is query_lens.dtype is block_table.dtype
              is free_pages.dtype is free_count.dtype is _I32
              and context_lens.get_device() == query_lens.get_device() == free_pages.get_device()
              == free_count.get_device() == dev
              and context_lens.shape == query_lens.shape == (R,) and free_count.shape == (1,)
              and free_pages.ndim == 1 and context_lens.is_contiguous()
              and query_lens.is_contiguous() and block_table.is_contiguous()
              and free_pages.is_contiguous() and 0 <= max_tokens < _LIM and 0 <= page_size < _LIM
              and 0 <= n_pages < _LIM)
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _explain("context_lens, query_lens and block_table must have the same number of requests, "
                 "free_count one element, and page_size, max_tokens and n_pages lie in [0, 2^31)",
                 (context_lens, "context_lens", _I32, 1), (query_lens, "query_lens", _I32, 1),
                 (block_table, "block_table", _I32, 2), (free_pages, "free_pages", _I32, 1),
                 (free_count, "free_count", _I32, 1))
    N = int(max_tokens)
    # One allocation: seq_lens, cu_query, token_req, positions, slot_mapping,
    # and the count and table unless they are updated in place.  The kernel is
    # launched before the tensors over its parts are made ("unsafe": not as
    # views that autograd would follow, which these integers need not be).
    sizes = [R, R + 1, N, N, N] if inplace else [R, R + 1, N, N, N, 1, R * W]
    base = torch.empty(sum(sizes), dtype=_I32, device=dev)
    at = base.data_ptr()
    tok = at + 8 * R + 4
    end = tok + 12 * N
    _call("smqa_paged_plan", dev, _lib.load().smqa_paged_plan, context_lens.data_ptr(),
          query_lens.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(),
          free_count.data_ptr(), R, W, int(page_size), int(n_pages), free_pages.shape[0], N,
          block_table.data_ptr() if inplace else end + 4,
          free_count.data_ptr() if inplace else end, at, at + 4 * R, tok, tok + 4 * N, tok + 8 * N)
    if inplace:
        table, count = block_table, free_count
        seq, cu, req, pos, slot = torch.unsafe_split_with_sizes(base, sizes)
    else:
        seq, cu, req, pos, slot, count, table = torch.unsafe_split_with_sizes(base, sizes)
        table = table.view(R, W)
    return PagedPlan(table, count, seq, cu, req, pos, slot)


def paged_release(block_table: torch.Tensor, release: torch.Tensor, free_pages: torch.Tensor,
                  free_count: torch.Tensor, n_pages: int,
                  seq_lens: Optional[torch.Tensor] = None) -> None:
    """Gives back the pages of the requests r with release[r] (bool [R]): in
    place, their block_table entries in [0, n_pages) go on the stack
    (free_pages, free_count) and become -1; their seq_lens, if given, 0."""
    tensors = [(block_table, "block_table", _I32, 2), (release, "release", torch.bool, 1),
               (free_pages, "free_pages", _I32, 1), (free_count, "free_count", _I32, 1)]
    if seq_lens is not None:
        tensors.append((seq_lens, "seq_lens", _I32, 1))
    for t in tensors:
        _need(*t)
    R, W = block_table.shape
    if release.shape[0] != R or free_count.shape[0] != 1 or \
            (seq_lens is not None and seq_lens.shape[0] != R) or \
            len({t.device for t, *_ in tensors}) != 1 or not 0 <= n_pages < _LIM:
        _explain(f"release and seq_lens must have R={R} entries, free_count one element, and n_pages "
                 "lie in [0, 2^31)", *tensors)
    _call("smqa_paged_release", block_table.get_device(), _lib.load().smqa_paged_release,
          block_table.data_ptr(), None if seq_lens is None else seq_lens.data_ptr(),
          release.data_ptr(), R, W, int(n_pages), free_pages.data_ptr(), free_count.data_ptr(),
          free_pages.shape[0])


def paged_kv_append(kv_new: torch.Tensor, slot_mapping: torch.Tensor, kv_cache: torch.Tensor,
                    kv_scales: torch.Tensor, positions: Optional[torch.Tensor] = None,
                    cos_sin: Optional[torch.Tensor] = None, rope_offset: Optional[int] = None,
                    interleaved: bool = False) -> tuple[torch.Tensor, torch.Tensor]:
    """Writes kv_new [T, D] bf16 into the cache at slot_mapping [T] int32 (C
    ABI ``smqa_paged_append``, ``smqa_paged_append_rope``); -1 skips a row.  In
    place; returns (kv_cache, kv_scales).  D is 64 or 512, or 128 for the
    indexer's keys.

    A page's scale is the smallest power of two that keeps its values within
    e4m3's 448; it grows while the page fills (the page's older rows are
    rescaled) and starts afresh when the page's first row is written.  The rows
    of one page must be consecutive, with slots ascending by one, as
    paged_plan lists them; a page listed otherwise (a slot twice, its rows apart)
    gets undefined codes and scale, the other pages theirs.

    With ``cos_sin`` [rows, rope_dim] fp32 (the cosines of a position's
    rope_dim/2 angles, then their sines) and ``positions`` [T] int32 the rows are
    rotated on the way, in fp32: rope_dim elements from ``rope_offset`` on (None:
    the last ones), in pairs of neighbours (``interleaved``) or rope_dim/2 apart.
    A position outside the table makes its row's rotated elements NaN."""
    rope = cos_sin is not None
    try:
        dev = kv_cache.get_device()
        n_pages, page_size, D = kv_cache.shape
        T = kv_new.shape[0]
        ok = (dev >= 0 and kv_cache.dtype is _E4M3 and kv_scales.dtype is _F32
              and kv_new.dtype is _BF16 and slot_mapping.dtype is _I32
              and kv_scales.get_device() == kv_new.get_device() == slot_mapping.get_device() == dev
              and kv_scales.shape == (n_pages,) and kv_new.shape == (T, D)
              and slot_mapping.shape == (T,) and kv_cache.is_contiguous()
              and kv_scales.is_contiguous() and kv_new.is_contiguous()
              and slot_mapping.is_contiguous())
        if rope and ok:
            rows, dim = cos_sin.shape
            offset = D - dim if rope_offset is None else rope_offset
            ok = (cos_sin.dtype is _F32 and positions.dtype is _I32
                  and cos_sin.get_device() == positions.get_device() == dev
                  and positions.shape == (T,) and cos_sin.is_contiguous()
                  and positions.is_contiguous() and dim > 0 and 0 <= offset < _LIM and rows < _LIM)
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok or (not rope and (positions is not None or rope_offset is not None)):
        more = [(positions, "positions", _I32, 1), (cos_sin, "cos_sin", _F32, 2)]
        _explain("kv_cache [n_pages,page_size,D], kv_scales [n_pages], kv_new [T,D], "
                 "slot_mapping [T], positions [T] and cos_sin [rows, 1 <= rope_dim <= D] (both or "
                 "neither, rope_offset >= 0 only with them) do not have matching shapes",
                 (kv_cache, "kv_cache", _E4M3, 3), (kv_scales, "kv_scales", _F32, 1),
                 (kv_new, "kv_new", _BF16, 2), (slot_mapping, "slot_mapping", _I32, 1),
                 *(more if rope else []))
    if rope:
        _call("smqa_paged_append_rope", dev, _lib.load().smqa_paged_append_rope, kv_new.data_ptr(),
              slot_mapping.data_ptr(), positions.data_ptr(), cos_sin.data_ptr(), T, D, page_size,
              n_pages, rows, dim, offset, bool(interleaved), kv_cache.data_ptr(),
              kv_scales.data_ptr())
    elif D == 128:
        _call("smqa_paged_append_rope", dev, _lib.load().smqa_paged_append_rope, kv_new.data_ptr(),
              slot_mapping.data_ptr(), None, None, T, D, page_size, n_pages, 0, 0, 0, 0,
              kv_cache.data_ptr(), kv_scales.data_ptr())
    else:
        _call("smqa_paged_append", dev, _lib.load().smqa_paged_append, kv_new.data_ptr(),
              slot_mapping.data_ptr(), T, D, page_size, n_pages, kv_cache.data_ptr(),
              kv_scales.data_ptr())
    return kv_cache, kv_scales


def paged_fwd_workspace_bytes(shape: _lib.PagedShape) -> int:
    return int(_lib.load().smqa_paged_fwd_workspace_bytes(shape))


def sparse_mqa_paged_fwd(q: torch.Tensor, kv_cache: torch.Tensor, kv_scales: torch.Tensor,
                         attn_sink: torch.Tensor, block_table: torch.Tensor,
                         seq_lens: torch.Tensor, token_req: torch.Tensor,
                         positions: Optional[torch.Tensor] = None,
                         topk_idxs: Optional[torch.Tensor] = None,
                         sm_scale: Optional[float] = None,
                         out: Optional[tuple[torch.Tensor, torch.Tensor]] = None,
                         workspace: Optional[torch.Tensor] = None, check_status: bool = False
                         ) -> tuple[torch.Tensor, torch.Tensor]:
    """Sparse MQA over the 8-bit paged cache, for single tokens and prompts.

    q [T,H,D] bf16, kv_cache [n_pages,page_size,D] float8_e4m3fn, kv_scales
    [n_pages] fp32, attn_sink [H] fp32, block_table [R,max_pages] and seq_lens
    [R] int32; token_req [T] int32 names each token's request (outside [0,R):
    padding).  With topk_idxs [T,topk] int32 a token attends to those positions
    of its request (entries outside [0, seq_len) are masked); without it, to
    every position up to its own, positions [T] int32.  Returns O [T,H,D] bf16
    and the log2 LSE [T,H] fp32 of sparse_mqa_fwd_interface.

    ``out`` = (o, lse) takes the results; rows of padding tokens are then left
    as they were, in fresh tensors they are O = 0 and LSE = -inf.
    ``workspace`` (uint8 CUDA tensor) is reused when large enough.  With
    ``check_status`` the call synchronizes and raises SMQAError
    (SMQA_ERR_DEVICE_TIMEOUT) if a kernel's bounded wait ran out.
    """
    try:
        dev = q.get_device()
        T, H, D = q.shape
        n_pages, page_size, _ = kv_cache.shape
        R, W = block_table.shape
        topk = 0 if topk_idxs is None else topk_idxs.shape[1]
        ok = (dev >= 0 and q.dtype is _BF16 and kv_cache.dtype is _E4M3
              and kv_scales.dtype is attn_sink.dtype is _F32
              and block_table.dtype is seq_lens.dtype is token_req.dtype is _I32
              and kv_cache.get_device() == kv_scales.get_device() == attn_sink.get_device()
              == block_table.get_device() == seq_lens.get_device() == token_req.get_device() == dev
              and kv_cache.shape[2] == D and kv_scales.shape == (n_pages,)
              and attn_sink.shape == (H,) and seq_lens.shape == (R,) and token_req.shape == (T,)
              and q.is_contiguous() and kv_cache.is_contiguous() and kv_scales.is_contiguous()
              and attn_sink.is_contiguous() and block_table.is_contiguous()
              and seq_lens.is_contiguous() and token_req.is_contiguous()
              and (topk_idxs is not None or positions is not None)
              and (positions is None or (
                  positions.dtype is _I32 and positions.get_device() == dev
                  and positions.shape == (T,) and positions.is_contiguous()))
              and (topk_idxs is None or (
                  topk_idxs.dtype is _I32 and topk_idxs.get_device() == dev and topk > 0
                  and topk_idxs.shape == (T, topk) and topk_idxs.is_contiguous()))
              and (workspace is None or (
                  workspace.dtype is torch.uint8 and workspace.get_device() == dev
                  and workspace.ndim == 1 and workspace.is_contiguous())))
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        more = [(positions, "positions", _I32, 1), (topk_idxs, "topk_idxs", _I32, 2),
                (workspace, "workspace", torch.uint8, 1)]
        _explain("q [T,H,D], kv_cache [n_pages,page_size,D], kv_scales [n_pages], attn_sink [H], "
                 "block_table [R,max_pages], seq_lens [R], token_req [T] and positions [T] or "
                 "topk_idxs [T,topk >= 1] (one of them is needed) do not have matching shapes",
                 (q, "q", _BF16, 3), (kv_cache, "kv_cache", _E4M3, 3),
                 (kv_scales, "kv_scales", _F32, 1), (attn_sink, "attn_sink", _F32, 1),
                 (block_table, "block_table", _I32, 2), (seq_lens, "seq_lens", _I32, 1),
                 (token_req, "token_req", _I32, 1), *[t for t in more if t[0] is not None])
    scale = D ** -0.5 if sm_scale is None else _scale(sm_scale, D)
    shp = _lib.PagedShape(T, R, H, D, topk, page_size, W, n_pages)
    lib = _lib.load()
    need = lib.smqa_paged_fwd_workspace_bytes(shp)
    if need > 0 and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((T, H), dtype=_F32, device=dev)
        flags = _lib.FLAG_ZERO_PADDING
    else:
        o, lse = out
        _need(o, "out[0]", _BF16, 3)
        _need(lse, "out[1]", _F32, 2)
        if o.shape != q.shape or lse.shape != (T, H) or o.device != q.device or \
                lse.device != q.device:
            raise ValueError("out must be (o like q, lse [T,H]) on q's device")
        flags = 0
    _call("smqa_paged_fwd", dev, lib.smqa_paged_fwd, q.data_ptr(), kv_cache.data_ptr(),
          kv_scales.data_ptr(), attn_sink.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
          token_req.data_ptr(), None if positions is None else positions.data_ptr(),
          None if topk_idxs is None else topk_idxs.data_ptr(), shp, scale, o.data_ptr(),
          lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.numel(), flags)
    if check_status:
        _check_device(q.device, "smqa_paged_fwd")
    return o, lse

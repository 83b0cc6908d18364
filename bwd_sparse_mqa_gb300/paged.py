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


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _same_device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> torch.device:
    dev = first.device
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must be on the same device")
    return dev


def _call(fn: str, device: torch.device, f, *args) -> None:
    """f(*args, current stream of ``device``) with that device current."""
    if torch.cuda.current_device() == device.index:
        st = f(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        with torch.cuda.device(device):
            st = f(*args, torch.cuda.current_stream(device).cuda_stream)
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
    _need(context_lens, "context_lens", torch.int32, 1)
    _need(query_lens, "query_lens", torch.int32, 1)
    _need(block_table, "block_table", torch.int32, 2)
    _need(free_pages, "free_pages", torch.int32, 1)
    _need(free_count, "free_count", torch.int32, 1)
    R, W = block_table.shape
    if context_lens.shape[0] != R or query_lens.shape[0] != R or free_count.shape[0] != 1:
        raise ValueError("context_lens, query_lens and block_table must have the same number of "
                         "requests, free_count one element")
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    dev = _same_device(context_lens, query_lens, block_table, free_pages, free_count)
    N = int(max_tokens)
    # One allocation: seq_lens, cu_query, token_req, positions, slot_mapping,
    # and the table and count unless they are updated in place.
    sizes = [R, R + 1, N, N, N] + ([] if inplace else [R * W, 1])
    out = torch.empty(sum(sizes), dtype=torch.int32, device=dev).split(sizes)
    table_out, count_out = (block_table, free_count) if inplace else (out[5].view(R, W), out[6])
    plan = PagedPlan(table_out, count_out, *out[:5])
    _call("smqa_paged_plan", dev, _lib.load().smqa_paged_plan, _ptr(context_lens),
          _ptr(query_lens), _ptr(block_table), _ptr(free_pages), _ptr(free_count), R, W,
          int(page_size), int(n_pages), free_pages.shape[0], N, _ptr(plan.block_table),
          _ptr(plan.free_count), _ptr(plan.seq_lens), _ptr(plan.cu_query), _ptr(plan.token_req),
          _ptr(plan.positions), _ptr(plan.slot_mapping))
    return plan


def paged_release(block_table: torch.Tensor, release: torch.Tensor, free_pages: torch.Tensor,
                  free_count: torch.Tensor, n_pages: int,
                  seq_lens: Optional[torch.Tensor] = None) -> None:
    """Gives back the pages of the requests r with release[r] (bool [R]): in
    place, their block_table entries in [0, n_pages) go on the stack
    (free_pages, free_count) and become -1; their seq_lens, if given, 0."""
    _need(block_table, "block_table", torch.int32, 2)
    _need(release, "release", torch.bool, 1)
    _need(free_pages, "free_pages", torch.int32, 1)
    _need(free_count, "free_count", torch.int32, 1)
    R, W = block_table.shape
    if seq_lens is not None:
        _need(seq_lens, "seq_lens", torch.int32, 1)
        if seq_lens.shape[0] != R:
            raise ValueError(f"seq_lens must have R={R} entries")
    if release.shape[0] != R or free_count.shape[0] != 1:
        raise ValueError(f"release must have R={R} entries, free_count one element")
    dev = _same_device(block_table, release, free_pages, free_count, seq_lens)
    _call("smqa_paged_release", dev, _lib.load().smqa_paged_release, _ptr(block_table),
          _ptr(seq_lens), _ptr(release), R, W, int(n_pages), _ptr(free_pages), _ptr(free_count),
          free_pages.shape[0])


def _need_cache(kv_cache: torch.Tensor, kv_scales: torch.Tensor) -> tuple:
    _need(kv_cache, "kv_cache", torch.float8_e4m3fn, 3)
    _need(kv_scales, "kv_scales", torch.float32, 1)
    if kv_scales.shape[0] != kv_cache.shape[0]:
        raise ValueError("kv_scales must have one entry per page of kv_cache")
    return kv_cache.shape


def paged_kv_append(kv_new: torch.Tensor, slot_mapping: torch.Tensor, kv_cache: torch.Tensor,
                    kv_scales: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Writes kv_new [T, D] bf16 into the cache at slot_mapping [T] int32 (C
    ABI ``smqa_paged_append``); -1 skips a row.  In place; returns (kv_cache,
    kv_scales).

    A page's scale is the smallest power of two that keeps its values within
    e4m3's 448; it grows while the page fills (the page's older rows are
    rescaled) and starts afresh when the page's first row is written.  The rows
    of one page must be consecutive, with slots ascending by one, as
    paged_plan lists them."""
    n_pages, page_size, D = _need_cache(kv_cache, kv_scales)
    _need(kv_new, "kv_new", torch.bfloat16, 2)
    _need(slot_mapping, "slot_mapping", torch.int32, 1)
    T = kv_new.shape[0]
    if kv_new.shape[1] != D or slot_mapping.shape[0] != T:
        raise ValueError(f"kv_new {tuple(kv_new.shape)} does not match kv_cache "
                         f"{tuple(kv_cache.shape)} and slot_mapping {tuple(slot_mapping.shape)}")
    dev = _same_device(kv_cache, kv_scales, kv_new, slot_mapping)
    _call("smqa_paged_append", dev, _lib.load().smqa_paged_append, _ptr(kv_new),
          _ptr(slot_mapping), T, D, page_size, n_pages, _ptr(kv_cache), _ptr(kv_scales))
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
    _need(q, "q", torch.bfloat16, 3)
    n_pages, page_size, D = _need_cache(kv_cache, kv_scales)
    _need(attn_sink, "attn_sink", torch.float32, 1)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(token_req, "token_req", torch.int32, 1)
    T, H, Dq = q.shape
    R, W = block_table.shape
    if Dq != D or attn_sink.shape[0] != H or seq_lens.shape[0] != R or token_req.shape[0] != T:
        raise ValueError("q, kv_cache, attn_sink, block_table, seq_lens and token_req do not have "
                         "matching shapes")
    topk = 0
    if positions is not None:
        _need(positions, "positions", torch.int32, 1)
        if positions.shape[0] != T:
            raise ValueError(f"positions must have T={T} entries")
    if topk_idxs is not None:
        _need(topk_idxs, "topk_idxs", torch.int32, 2)
        topk = topk_idxs.shape[1]
        if topk_idxs.shape[0] != T or topk == 0:
            raise ValueError(f"topk_idxs must be [T={T}, topk >= 1]")
    elif positions is None:
        raise ValueError("positions is needed without topk_idxs")
    dev = _same_device(q, kv_cache, kv_scales, attn_sink, block_table, seq_lens, token_req,
                       positions, topk_idxs, workspace)
    scale = _scale(sm_scale, D)
    shp = _lib.PagedShape(T, R, H, D, topk, page_size, W, n_pages)
    lib = _lib.load()
    need = lib.smqa_paged_fwd_workspace_bytes(shp)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1)
    if need > 0 and (workspace is None or workspace.numel() < need):
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if out is None:
        o = torch.empty_like(q)
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
        flags = _lib.FLAG_ZERO_PADDING
    else:
        o, lse = out
        _need(o, "out[0]", torch.bfloat16, 3)
        _need(lse, "out[1]", torch.float32, 2)
        if o.shape != q.shape or tuple(lse.shape) != (T, H):
            raise ValueError("out must be (o like q, lse [T,H])")
        _same_device(q, o, lse)
        flags = 0
    _call("smqa_paged_fwd", dev, lib.smqa_paged_fwd, _ptr(q), _ptr(kv_cache), _ptr(kv_scales),
          _ptr(attn_sink), _ptr(block_table), _ptr(seq_lens), _ptr(token_req), _ptr(positions),
          _ptr(topk_idxs), shp, scale, _ptr(o), _ptr(lse), _ptr(workspace),
          0 if workspace is None else workspace.numel(), flags)
    if check_status:
        _check_device(dev, "smqa_paged_fwd")
    return o, lse

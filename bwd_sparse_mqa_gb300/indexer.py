"""The lightning indexer: which positions sparse MQA attends to, and its training.

A token's score of a key row is sum_h weights[h] ReLU(index_q[h] . index_k); the
blocks with the best rows give the ``topk_idxs`` of sparse_mqa (contiguous keys,
``indexer_topk``) and of sparse_mqa_paged_fwd (keys in an 8-bit paged cache,
``paged_indexer_topk``).  A layer of a prompt or of a training step is

    idx = indexer_topk(index_q, weights, index_k, topk)
    o, lse = sparse_mqa(q, kv, attn_sink, idx)
    scores = indexer_scores(index_q, weights, index_k, idx)   # differentiable, -inf where masked

and of a server's step, behind paged_plan,

    paged_kv_append(kv_new, plan.slot_mapping, kv_cache, kv_scales, plan.positions, cos_sin)
    paged_kv_append(k_new, plan.slot_mapping, k_cache, k_scales, plan.positions, cos_sin)
    idx = paged_indexer_topk(index_q, weights, k_cache, k_scales, plan.block_table,
                             plan.seq_lens, plan.token_req, plan.positions, topk)
    o, lse = sparse_mqa_paged_fwd(q, kv_cache, kv_scales, attn_sink, plan.block_table,
                                  plan.seq_lens, plan.token_req, plan.positions, idx)

Every call is asynchronous on the current stream of its tensors' device, reads
nothing back to the host and can be captured in a CUDA graph.  As in api.py,
PyTorch only supplies device memory and the stream; there is no CPU path.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .api import _check_device, _need
from .paged import _BF16, _E4M3, _F32, _I32, _LIM, _call, _explain


def _buffers(need: int, workspace: Optional[torch.Tensor], out: Optional[torch.Tensor],
             shape: tuple, dev: int) -> tuple[torch.Tensor, torch.Tensor]:
    """Workspace of ``need`` bytes and the int32 output, the given ones where they will do."""
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1)
        if workspace.get_device() != dev:
            raise ValueError("workspace must be on the tensors' device")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty(shape, dtype=_I32, device=dev)
    else:
        _need(out, "out", _I32, len(shape))
        if out.shape != shape or out.get_device() != dev:
            raise ValueError(f"out must be {list(shape)} on the tensors' device")
    return workspace, out


def _int32(**sizes: int) -> None:
    for name, v in sizes.items():
        if not -_LIM <= v < _LIM:
            raise ValueError(f"{name} must lie within 32 bits")


def indexer_topk_workspace_bytes(shape: _lib.Shape, block_size: int = 1) -> int:
    return int(_lib.load().smqa_indexer_topk_workspace_bytes(shape, block_size))


def indexer_topk(index_q: torch.Tensor, weights: torch.Tensor, index_k: torch.Tensor, topk: int,
                 block_size: int = 1, recent: int = 0, first_position: Optional[int] = None,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 check_status: bool = False) -> torch.Tensor:
    """The positions each token attends to (C ABI ``smqa_indexer_topk``).

    index_q [B,S,H,D] bf16, weights [B,S,H] fp32, index_k [B,S_kv,D] bf16.  Query
    s stands at ``first_position`` + s (None: S_kv - S, the last S positions of a
    causal sequence; S_kv or more: every query sees every row) and ranks the rows
    up to there by sum_h weights[h] ReLU(index_q[h] . index_k[j]); blocks of
    ``block_size`` positions rank by their best row.  The last ``recent`` positions
    a query sees always are among its choice.  Returns topk_idxs [B,S,topk] int32:
    the topk / block_size best blocks' positions, ascending, then -1.  The choice
    is that of the scores as real numbers, ties to the lowest block (scores closer
    than 2^-40 sum_h |w_h||q_h||k_j| may count as equal; the C header has the limits
    of magnitudes).

    ``out`` takes the result, ``workspace`` (uint8 CUDA tensor) is reused when
    large enough.  With ``check_status`` the call synchronizes and raises
    SMQAError (SMQA_ERR_DEVICE_TIMEOUT) if a kernel's bounded wait ran out.
    """
    try:
        dev = index_q.get_device()
        B, S, H, D = index_q.shape
        S_kv = index_k.shape[1]
        ok = (dev >= 0 and index_q.dtype is index_k.dtype is _BF16 and weights.dtype is _F32
              and weights.get_device() == index_k.get_device() == dev
              and weights.shape == (B, S, H) and index_k.shape == (B, S_kv, D)
              and index_q.is_contiguous() and weights.is_contiguous() and index_k.is_contiguous())
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _explain("index_q [B,S,H,D], weights [B,S,H] and index_k [B,S_kv,D] do not have matching "
                 "shapes", (index_q, "index_q", _BF16, 4), (weights, "weights", _F32, 3),
                 (index_k, "index_k", _BF16, 3))
    _int32(topk=topk, block_size=block_size, recent=recent)
    first = S_kv - S if first_position is None else int(first_position)
    first = max(-2 * _LIM, min(2 * _LIM, first))
    shp = _lib.Shape(B, S, S_kv, H, D, topk)
    lib = _lib.load()
    workspace, out = _buffers(lib.smqa_indexer_topk_workspace_bytes(shp, block_size), workspace, out,
                              (B, S, max(topk, 0)), dev)
    _call("smqa_indexer_topk", dev, lib.smqa_indexer_topk, index_q.data_ptr(), weights.data_ptr(),
          index_k.data_ptr(), shp, block_size, recent, first, out.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    if check_status:
        _check_device(index_q.device, "smqa_indexer_topk")
    return out


def paged_indexer_topk_workspace_bytes(shape: _lib.PagedShape, block_size: int = 1) -> int:
    return int(_lib.load().smqa_paged_indexer_topk_workspace_bytes(shape, block_size))


def paged_indexer_topk(index_q: torch.Tensor, weights: torch.Tensor, k_cache: torch.Tensor,
                       k_scales: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                       token_req: torch.Tensor, positions: Optional[torch.Tensor], topk: int,
                       block_size: int = 1, recent: int = 0, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, check_status: bool = False
                       ) -> torch.Tensor:
    """indexer_topk over index keys in an 8-bit paged cache, for single tokens and
    prompts (C ABI ``smqa_paged_indexer_topk``).

    index_q [T,H,D] bf16, weights [T,H] fp32, k_cache [n_pages,page_size,D]
    float8_e4m3fn and k_scales [n_pages] fp32 as paged_kv_append writes them;
    block_table [R,max_pages], seq_lens [R], token_req [T] and positions [T] int32
    as in sparse_mqa_paged_fwd: a token sees its request's positions up to its own
    (``positions`` None: all of them), on pages that the table has.  Returns
    topk_idxs [T,topk] int32, positions in the token's own request, ascending,
    then -1.

    With ``out``, rows of padding tokens are left as they were, in a fresh tensor
    they are -1.  ``workspace`` and ``check_status`` as in indexer_topk.  The
    workspace and the number of launches follow the table's width: where it is far
    wider than the longest request, a narrower copy makes prompts faster.
    """
    try:
        dev = index_q.get_device()
        T, H, D = index_q.shape
        n_pages, page_size, _ = k_cache.shape
        R, W = block_table.shape
        ok = (dev >= 0 and index_q.dtype is _BF16 and k_cache.dtype is _E4M3
              and weights.dtype is k_scales.dtype is _F32
              and block_table.dtype is seq_lens.dtype is token_req.dtype is _I32
              and weights.get_device() == k_cache.get_device() == k_scales.get_device()
              == block_table.get_device() == seq_lens.get_device() == token_req.get_device() == dev
              and weights.shape == (T, H) and k_cache.shape[2] == D and k_scales.shape == (n_pages,)
              and seq_lens.shape == (R,) and token_req.shape == (T,) and index_q.is_contiguous()
              and weights.is_contiguous() and k_cache.is_contiguous() and k_scales.is_contiguous()
              and block_table.is_contiguous() and seq_lens.is_contiguous()
              and token_req.is_contiguous()
              and (positions is None or (
                  positions.dtype is _I32 and positions.get_device() == dev
                  and positions.shape == (T,) and positions.is_contiguous())))
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        more = [] if positions is None else [(positions, "positions", _I32, 1)]
        _explain("index_q [T,H,D], weights [T,H], k_cache [n_pages,page_size,D], k_scales [n_pages], "
                 "block_table [R,max_pages], seq_lens [R], token_req [T] and positions [T] do not "
                 "have matching shapes", (index_q, "index_q", _BF16, 3), (weights, "weights", _F32, 2),
                 (k_cache, "k_cache", _E4M3, 3), (k_scales, "k_scales", _F32, 1),
                 (block_table, "block_table", _I32, 2), (seq_lens, "seq_lens", _I32, 1),
                 (token_req, "token_req", _I32, 1), *more)
    _int32(topk=topk, block_size=block_size, recent=recent)
    shp = _lib.PagedShape(T, R, H, D, topk, page_size, W, n_pages)
    lib = _lib.load()
    flags = _lib.FLAG_ZERO_PADDING if out is None else 0
    workspace, out = _buffers(lib.smqa_paged_indexer_topk_workspace_bytes(shp, block_size), workspace,
                              out, (T, max(topk, 0)), dev)
    _call("smqa_paged_indexer_topk", dev, lib.smqa_paged_indexer_topk, index_q.data_ptr(),
          weights.data_ptr(), k_cache.data_ptr(), k_scales.data_ptr(), block_table.data_ptr(),
          seq_lens.data_ptr(), token_req.data_ptr(),
          None if positions is None else positions.data_ptr(), shp, block_size, recent,
          out.data_ptr(), workspace.data_ptr(), workspace.numel(), flags)
    if check_status:
        _check_device(index_q.device, "smqa_paged_indexer_topk")
    return out


def _scores_args(index_q, weights, index_k, topk_indices):
    """(device, shape) of checked arguments."""
    try:
        dev = index_q.get_device()
        B, S, H, D = index_q.shape
        S_kv, topk = index_k.shape[1], topk_indices.shape[2]
        ok = (dev >= 0 and index_q.dtype is index_k.dtype is _BF16 and weights.dtype is _F32
              and topk_indices.dtype is _I32 and weights.get_device() == index_k.get_device()
              == topk_indices.get_device() == dev and weights.shape == (B, S, H)
              and index_k.shape == (B, S_kv, D) and topk_indices.shape == (B, S, topk)
              and index_q.is_contiguous() and weights.is_contiguous() and index_k.is_contiguous()
              and topk_indices.is_contiguous())
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        _explain("index_q [B,S,H,D], weights [B,S,H], index_k [B,S_kv,D] and topk_indices [B,S,topk] "
                 "do not have matching shapes", (index_q, "index_q", _BF16, 4),
                 (weights, "weights", _F32, 3), (index_k, "index_k", _BF16, 3),
                 (topk_indices, "topk_indices", _I32, 3))
    return dev, _lib.Shape(B, S, S_kv, H, D, topk)


def indexer_scores_fwd(index_q: torch.Tensor, weights: torch.Tensor, index_k: torch.Tensor,
                       topk_indices: torch.Tensor, check_status: bool = False) -> torch.Tensor:
    """The indexer's scores at topk_indices (C ABI ``smqa_indexer_scores``):
    scores[b,s,j] = sum_h weights[b,s,h] ReLU(index_q[b,s,h] . index_k[b,idx[b,s,j]]),
    -inf where an index lies outside [0,S_kv).

    index_q [B,S,H,D] bf16, weights [B,S,H] fp32, index_k [B,S_kv,D] bf16,
    topk_indices [B,S,topk] int32; returns scores [B,S,topk] fp32, freshly
    allocated.  ``check_status`` as in indexer_topk."""
    dev, shp = _scores_args(index_q, weights, index_k, topk_indices)
    scores = torch.empty((shp.B, shp.S, shp.topk), dtype=_F32, device=index_q.device)
    _call("smqa_indexer_scores", dev, _lib.load().smqa_indexer_scores, index_q.data_ptr(),
          weights.data_ptr(), index_k.data_ptr(), topk_indices.data_ptr(), shp, scores.data_ptr())
    if check_status:
        _check_device(index_q.device, "smqa_indexer_scores")
    return scores


def indexer_scores_bwd(index_q: torch.Tensor, weights: torch.Tensor, index_k: torch.Tensor,
                       topk_indices: torch.Tensor, grad_scores: torch.Tensor,
                       return_dk_accum_dtype: bool = False,
                       workspace: Optional[torch.Tensor] = None, check_status: bool = False
                       ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of indexer_scores_fwd for grad_scores [B,S,topk] fp32 (C ABI
    ``smqa_indexer_scores_bwd``): (dq like index_q, dweights [B,S,H] fp32, dindex_k
    like index_k, or fp32 with ``return_dk_accum_dtype``), freshly allocated.
    Masked slots' gradients are not looked at.  dindex_k is summed by fp32 atomics:
    its last bits may change from run to run.  ``workspace`` (uint8 CUDA tensor) is
    reused when large enough; ``check_status`` as in indexer_topk."""
    dev, shp = _scores_args(index_q, weights, index_k, topk_indices)
    _need(grad_scores, "grad_scores", _F32, 3)
    if grad_scores.shape != topk_indices.shape or grad_scores.get_device() != dev:
        raise ValueError("grad_scores must be like topk_indices, on the same device")
    lib = _lib.load()
    flags = _lib.FLAG_RETURN_DKV_FP32 if return_dk_accum_dtype else 0
    need = lib.smqa_indexer_scores_bwd_workspace_bytes(shp, flags)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1)
        if workspace.get_device() != dev:
            raise ValueError("workspace must be on the tensors' device")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=index_q.device)
    dq, dw = torch.empty_like(index_q), torch.empty_like(weights)
    dk = torch.empty_like(index_k, dtype=_F32 if return_dk_accum_dtype else _BF16)
    _call("smqa_indexer_scores_bwd", dev, lib.smqa_indexer_scores_bwd, index_q.data_ptr(),
          weights.data_ptr(), index_k.data_ptr(), topk_indices.data_ptr(), grad_scores.data_ptr(),
          shp, dq.data_ptr(), dw.data_ptr(), dk.data_ptr(), workspace.data_ptr() or None,
          workspace.numel(), flags)
    if check_status:
        _check_device(index_q.device, "smqa_indexer_scores_bwd")
    return dq, dw, dk


class IndexerScoresFunction(torch.autograd.Function):
    """Autograd around the scores' forward and backward kernels: gradients flow
    to index_q, weights and index_k."""

    @staticmethod
    def forward(ctx, index_q, weights, index_k, topk_indices, check_status=False):
        ctx.save_for_backward(index_q, weights, index_k, topk_indices)
        ctx.check_status = check_status
        return indexer_scores_fwd(index_q, weights, index_k, topk_indices, check_status)

    @staticmethod
    def backward(ctx, grad_scores):
        if torch.is_grad_enabled():                      # (the gradients would pass for constants)
            raise RuntimeError("indexer_scores is differentiable once (no create_graph)")
        index_q, weights, index_k, topk_indices = ctx.saved_tensors
        dq, dw, dk = indexer_scores_bwd(index_q, weights, index_k, topk_indices,
                                        grad_scores.to(_F32).contiguous(),
                                        check_status=ctx.check_status)
        return dq, dw, dk, None, None


def indexer_scores(index_q: torch.Tensor, weights: torch.Tensor, index_k: torch.Tensor,
                   topk_indices: torch.Tensor, check_status: bool = False) -> torch.Tensor:
    """Differentiable indexer_scores_fwd: gradients with respect to index_q, weights
    and index_k, once (create_graph raises).  With ``check_status`` the
    forward and the backward each synchronize and raise SMQAError if a kernel's
    bounded wait ran out.  A backward pass is captured with leaves that no other
    live graph holds: PyTorch adds a leaf's gradient on the stream of the graph that
    used it first."""
    return IndexerScoresFunction.apply(index_q, weights, index_k, topk_indices, check_status)

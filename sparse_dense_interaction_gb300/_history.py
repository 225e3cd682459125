"""ctypes binding of the event-history operators (C ABI:
``include/dlrm_history.h``).

Argument marshalling only, as in :mod:`._native`: the functions carry the C
names, take torch CUDA tensors of any strides with unit stride in the last
dimension, and raise :class:`DlrmError` on a non-zero status.  Token rows are
``[n][heads][d]``; a cache is a pair of ``[pages][page_size][heads][d]``
tensors or views (of a ``[pages][heads][page_size][d]`` tensor through
``transpose(1, 2)``); page tables are int32 ``[S][pages per sequence]``.
"""
from __future__ import annotations

import struct

import torch

from ._native import _TORCH_DTYPES, _check, _ptr, _stream, load

ROPE_HALF, ROPE_INTERLEAVED = 0, 1

# The C structs, packed: short calls are bound by the host, and a packed bytes
# object costs a third of a ctypes.Structure.
_HEADS = struct.Struct("@Pqqi4x").pack   # dlrm_heads: ptr, token_stride, head_stride, heads
_ROPE = struct.Struct("@PqPii").pack     # dlrm_rope: table, length, positions, rot, layout
_CACHE = struct.Struct("@PPqqqqii").pack  # dlrm_kv_cache: k, v, pages, three strides, page_size, heads
_BATCH = struct.Struct("@qqPPPqq").pack  # dlrm_kv_batch: S, n, offsets, lengths, page_table, stride, width


def _heads(t, n, d, dtype):
    """A dlrm_heads of ``t``, which must be [n][heads][d] of ``dtype``."""
    tokens, heads, width = t.shape
    token, head, unit = t.stride()
    if tokens != n or width != d or t.dtype is not dtype or not t.is_cuda or (unit != 1 and d > 1):
        raise ValueError("heads are [n][heads][d] CUDA tensors of one type, n and d, with unit stride in the last "
                         "dimension")
    return _HEADS(t.data_ptr(), token, head, heads)


def _weight(w, d):
    if w is None:
        return None
    if w.dtype is not torch.float32 or w.dim() != 1 or w.numel() != d or not w.is_cuda or not w.is_contiguous():
        raise ValueError("a norm's weight and its gradient are contiguous fp32 [d] CUDA tensors")
    return w.data_ptr()


def _int64(t, what, n):
    if t.dtype is not torch.int64 or t.dim() != 1 or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} is a contiguous int64 [{n}] CUDA tensor")
    return t.data_ptr()


def _workspace(t):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("a workspace is a contiguous CUDA tensor")
    return t.data_ptr()


def _flag(t):
    if t is None:
        return None
    if t.dtype is not torch.int32 or not t.is_cuda or t.numel() < 1:
        raise ValueError("err_flag is an int32 CUDA tensor")
    return t.data_ptr()


def _rope(rope, positions, interleaved, n):
    if rope is None:
        return None
    if rope.dtype is not torch.float32 or rope.dim() != 2 or not rope.is_cuda or not rope.is_contiguous():
        raise ValueError("rope is a contiguous fp32 [positions][rot] CUDA table")
    length, rot = rope.shape
    return _ROPE(rope.data_ptr(), length, 0 if positions is None else _int64(positions, "positions", n), rot,
                 ROPE_INTERLEAVED if interleaved else ROPE_HALF)


def _cache(k_cache, v_cache, d, dtype):
    strides = k_cache.stride()
    if v_cache.stride() != strides or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape and one set of strides")
    pages, page_size, heads, width = k_cache.shape
    page, slot, head, unit = strides
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype or width != d or (unit != 1 and d > 1) or not (
            k_cache.is_cuda and v_cache.is_cuda):
        raise ValueError("a cache is a pair of [pages][page_size][heads][d] CUDA tensors of the tokens' type, with "
                         "unit stride in the last dimension")
    return _CACHE(k_cache.data_ptr(), v_cache.data_ptr(), pages, page, slot, head, page_size, heads)


def _batch(offsets, lengths, page_table, n):
    S = lengths.numel()
    rows, width = page_table.shape
    stride, unit = page_table.stride()
    if page_table.dtype is not torch.int32 or rows != S or (unit != 1 and width > 1) or not page_table.is_cuda:
        raise ValueError("page_table is an int32 [S][pages] CUDA tensor with unit stride in its last dimension")
    return _BATCH(S, n, _int64(offsets, "offsets", S + 1), _int64(lengths, "lengths", S), page_table.data_ptr(),
                  stride, width)


def dlrm_qk_norm_rope_fwd(q, k, q_weight, k_weight, eps: float, rope, positions, q_out, k_out,
                          interleaved: bool = False, err_flag=None, stream=None):
    """Norms the heads of ``q`` [n][heads][d] and ``k`` (None: queries alone)
    and turns them by their positions, into ``q_out`` and ``k_out``.

    A weight is fp32 [d], or None for no norm; ``rope`` is an fp32
    [positions][rot] table of cosines, then sines, or None for no rotation;
    ``positions`` is int64 [n].  Pairs are (i, i + rot/2), or (2i, 2i + 1)
    with ``interleaved``."""
    n, _, d = q.shape
    dtype = q.dtype
    _check(load().dlrm_qk_norm_rope_fwd(
        _heads(q, n, d, dtype), None if k is None else _heads(k, n, d, dtype), n, d, _TORCH_DTYPES[dtype],
        _weight(q_weight, d), _weight(k_weight, d), eps, _rope(rope, positions, interleaved, n),
        _heads(q_out, n, d, dtype), None if k_out is None else _heads(k_out, n, d, dtype), _flag(err_flag),
        _stream(stream)), "dlrm_qk_norm_rope_fwd")


def dlrm_qk_norm_rope_bwd_workspace_size(n: int, q_heads: int, k_heads: int, d: int) -> int:
    return load().dlrm_qk_norm_rope_bwd_workspace_size(n, q_heads, k_heads, d)


def dlrm_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, eps: float, rope, positions, dq, dk, dq_weight,
                          dk_weight, workspace, interleaved: bool = False, err_flag=None, stream=None):
    """Gradients of :func:`dlrm_qk_norm_rope_fwd` into ``dq``, ``dk`` and, where
    not None, ``dq_weight`` and ``dk_weight`` (fp32 [d]); ``workspace`` is a
    uint8 tensor of :func:`dlrm_qk_norm_rope_bwd_workspace_size` bytes."""
    n, _, d = q.shape
    dtype = q.dtype
    _check(load().dlrm_qk_norm_rope_bwd(
        _heads(dq_out, n, d, dtype), None if dk_out is None else _heads(dk_out, n, d, dtype), _heads(q, n, d, dtype),
        None if k is None else _heads(k, n, d, dtype), n, d, _TORCH_DTYPES[dtype], _weight(q_weight, d),
        _weight(k_weight, d), eps, _rope(rope, positions, interleaved, n), _heads(dq, n, d, dtype),
        None if dk is None else _heads(dk, n, d, dtype), _weight(dq_weight, d), _weight(dk_weight, d),
        _workspace(workspace), workspace.nbytes, _flag(err_flag), _stream(stream)), "dlrm_qk_norm_rope_bwd")


def dlrm_kv_append(k, v, offsets, lengths, page_table, k_cache, v_cache, k_weight=None, eps: float = 1e-6, rope=None,
                   positions=None, interleaved: bool = False, q=None, q_weight=None, q_out=None, err_flag=None,
                   stream=None):
    """Stores the new tokens' keys (normed with ``k_weight``, turned) and values
    in the cache, at the ends of the histories of ``lengths`` tokens; with
    ``q`` and ``q_out`` the queries are normed and turned too.  The rotation
    is by a token's place in its history unless ``positions`` are given."""
    n, _, d = k.shape
    dtype = k.dtype
    _check(load().dlrm_kv_append(
        _heads(k, n, d, dtype), _heads(v, n, d, dtype), _batch(offsets, lengths, page_table, n),
        _cache(k_cache, v_cache, d, dtype), d, _TORCH_DTYPES[dtype], _weight(k_weight, d), eps,
        _rope(rope, positions, interleaved, n), None if q is None else _heads(q, n, d, dtype), _weight(q_weight, d),
        None if q_out is None else _heads(q_out, n, d, dtype), _flag(err_flag), _stream(stream)), "dlrm_kv_append")


def dlrm_kv_attn_workspace_size(S: int, n: int, q_heads: int, kv_heads: int, d: int, max_new: int,
                                max_len: int) -> int:
    return load().dlrm_kv_attn_workspace_size(S, n, q_heads, kv_heads, d, max_new, max_len)


def dlrm_kv_attn_fwd(q, offsets, lengths, page_table, k_cache, v_cache, out, scale: float, workspace, max_new: int,
                     max_len: int, causal: bool = True, window: int = 0, lse=None, err_flag=None, stream=None):
    """Attention of the new tokens ``q`` [n][heads][d] over the cache into
    ``out`` (same shape); ``lse`` (optional) is a contiguous fp32 [n][heads].

    ``causal``: the queries are the last tokens of their histories and see
    those up to their own; else each sees the whole history.  ``window`` > 0
    keeps the last ``window`` of them.  ``max_new`` and ``max_len`` bound the
    batch's new tokens per sequence and lengths; ``workspace`` is a uint8
    tensor of :func:`dlrm_kv_attn_workspace_size` bytes."""
    n, heads, d = q.shape
    dtype = q.dtype
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (n, heads) or not lse.is_cuda
                            or not lse.is_contiguous()):
        raise ValueError("lse is a contiguous fp32 [n][heads] CUDA tensor")
    _check(load().dlrm_kv_attn_fwd(
        _heads(q, n, d, dtype), _batch(offsets, lengths, page_table, n), _cache(k_cache, v_cache, d, dtype), d,
        _TORCH_DTYPES[dtype], scale, 1 if causal else 0, window, max_new, max_len, _heads(out, n, d, dtype),
        _ptr(lse), _workspace(workspace), workspace.nbytes, _flag(err_flag), _stream(stream)), "dlrm_kv_attn_fwd")

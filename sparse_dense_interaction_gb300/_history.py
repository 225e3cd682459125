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

import ctypes

import torch

from ._native import _TORCH_DTYPES, _check, _i32, _i64, _ptr, _stream, _vp, load

ROPE_HALF, ROPE_INTERLEAVED = 0, 1


class _Heads(ctypes.Structure):
    _fields_ = [("ptr", _vp), ("token_stride", _i64), ("head_stride", _i64), ("heads", _i32)]


class _Rope(ctypes.Structure):
    _fields_ = [("table", _vp), ("length", _i64), ("positions", _vp), ("rot", _i32), ("layout", _i32)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("pages", _i64), ("page_stride", _i64), ("slot_stride", _i64),
                ("head_stride", _i64), ("page_size", _i32), ("heads", _i32)]


class _Batch(ctypes.Structure):
    _fields_ = [("S", _i64), ("n", _i64), ("offsets", _vp), ("lengths", _vp), ("page_table", _vp),
                ("table_stride", _i64), ("table_width", _i64)]


def _heads(t, like):
    """A dlrm_heads of ``t`` [n][heads][d], with the type, tokens and width of ``like``."""
    n, heads, d = t.shape
    token, head, unit = t.stride()
    if not t.is_cuda or t.dtype != like.dtype or n != like.shape[0] or d != like.shape[2] or (unit != 1 and d > 1):
        raise ValueError("heads are [n][heads][d] CUDA tensors of one type, n and d, with unit stride in the last "
                         "dimension")
    return _Heads(t.data_ptr(), token, head, heads)


def _opt_heads(t, like):
    return None if t is None else ctypes.byref(_heads(t, like))


def _weight(w, d):
    if w is None:
        return None
    if not w.is_cuda or w.dtype != torch.float32 or w.shape != (d,) or (d > 1 and w.stride(0) != 1):
        raise ValueError("a norm's weight and its gradient are contiguous fp32 [d] CUDA tensors")
    return w.data_ptr()


def _int64(t, what, n):
    if not t.is_cuda or t.dtype != torch.int64 or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} is a contiguous int64 [{n}] CUDA tensor")
    return t.data_ptr()


def _rope(rope, positions, interleaved, n):
    if rope is None:
        return None
    if not rope.is_cuda or rope.dtype != torch.float32 or rope.dim() != 2 or not rope.is_contiguous():
        raise ValueError("rope is a contiguous fp32 [positions][rot] CUDA table")
    at = None if positions is None else _int64(positions, "positions", n)
    return ctypes.byref(_Rope(rope.data_ptr(), rope.shape[0], at, rope.shape[1],
                              ROPE_INTERLEAVED if interleaved else ROPE_HALF))


def _cache(k_cache, v_cache, like):
    if k_cache.stride() != v_cache.stride() or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape and one set of strides")
    pages, page_size, heads, d = k_cache.shape
    page, slot, head, unit = k_cache.stride()
    if not (k_cache.is_cuda and v_cache.is_cuda) or k_cache.dtype != like.dtype or v_cache.dtype != like.dtype or (
            d != like.shape[2] or (unit != 1 and d > 1)):
        raise ValueError("a cache is a pair of [pages][page_size][heads][d] CUDA tensors of the tokens' type, with "
                         "unit stride in the last dimension")
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), pages, page, slot, head, page_size, heads)


def _batch(offsets, lengths, page_table, n):
    S = lengths.shape[0]
    if not page_table.is_cuda or page_table.dtype != torch.int32 or page_table.dim() != 2 or (
            page_table.shape[0] != S or (page_table.shape[1] > 1 and page_table.stride(1) != 1)):
        raise ValueError("page_table is an int32 [S][pages] CUDA tensor with unit stride in its last dimension")
    return _Batch(S, n, _int64(offsets, "offsets", S + 1), _int64(lengths, "lengths", S), page_table.data_ptr(),
                  page_table.stride(0), page_table.shape[1])


def dlrm_qk_norm_rope_fwd(q, k, q_weight, k_weight, eps: float, rope, positions, q_out, k_out,
                          interleaved: bool = False, err_flag=None, stream=None):
    """Norms the heads of ``q`` [n][heads][d] and ``k`` (None: queries alone)
    and turns them by their positions, into ``q_out`` and ``k_out``.

    A weight is fp32 [d], or None for no norm; ``rope`` is an fp32
    [positions][rot] table of cosines, then sines, or None for no rotation;
    ``positions`` is int64 [n].  Pairs are (i, i + rot/2), or (2i, 2i + 1)
    with ``interleaved``."""
    n, _, d = q.shape
    _check(load().dlrm_qk_norm_rope_fwd(
        ctypes.byref(_heads(q, q)), _opt_heads(k, q), n, d, _TORCH_DTYPES[q.dtype], _weight(q_weight, d),
        _weight(k_weight, d), eps, _rope(rope, positions, interleaved, n), ctypes.byref(_heads(q_out, q)),
        _opt_heads(k_out, q), _ptr(err_flag), _stream(stream)), "dlrm_qk_norm_rope_fwd")


def dlrm_qk_norm_rope_bwd_workspace_size(n: int, q_heads: int, k_heads: int, d: int) -> int:
    return load().dlrm_qk_norm_rope_bwd_workspace_size(n, q_heads, k_heads, d)


def dlrm_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, eps: float, rope, positions, dq, dk, dq_weight,
                          dk_weight, workspace, interleaved: bool = False, err_flag=None, stream=None):
    """Gradients of :func:`dlrm_qk_norm_rope_fwd` into ``dq``, ``dk`` and, where
    not None, ``dq_weight`` and ``dk_weight`` (fp32 [d]); ``workspace`` is a
    uint8 tensor of :func:`dlrm_qk_norm_rope_bwd_workspace_size` bytes."""
    n, _, d = q.shape
    _check(load().dlrm_qk_norm_rope_bwd(
        ctypes.byref(_heads(dq_out, q)), _opt_heads(dk_out, q), ctypes.byref(_heads(q, q)), _opt_heads(k, q), n, d,
        _TORCH_DTYPES[q.dtype], _weight(q_weight, d), _weight(k_weight, d), eps,
        _rope(rope, positions, interleaved, n), ctypes.byref(_heads(dq, q)), _opt_heads(dk, q),
        _weight(dq_weight, d), _weight(dk_weight, d), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _ptr(err_flag), _stream(stream)), "dlrm_qk_norm_rope_bwd")


def dlrm_kv_append(k, v, offsets, lengths, page_table, k_cache, v_cache, k_weight=None, eps: float = 1e-6, rope=None,
                   positions=None, interleaved: bool = False, q=None, q_weight=None, q_out=None, err_flag=None,
                   stream=None):
    """Stores the new tokens' keys (normed with ``k_weight``, turned) and values
    in the cache, at the ends of the histories of ``lengths`` tokens; with
    ``q`` and ``q_out`` the queries are normed and turned too.  The rotation
    is by a token's place in its history unless ``positions`` are given."""
    n, _, d = k.shape
    batch = _batch(offsets, lengths, page_table, n)
    cache = _cache(k_cache, v_cache, k)
    _check(load().dlrm_kv_append(
        ctypes.byref(_heads(k, k)), ctypes.byref(_heads(v, k)), ctypes.byref(batch), ctypes.byref(cache), d,
        _TORCH_DTYPES[k.dtype], _weight(k_weight, d), eps, _rope(rope, positions, interleaved, n), _opt_heads(q, k),
        _weight(q_weight, d), _opt_heads(q_out, k), _ptr(err_flag), _stream(stream)), "dlrm_kv_append")


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
    if lse is not None and not (lse.is_cuda and lse.dtype == torch.float32 and lse.shape == (n, heads)
                                and lse.is_contiguous()):
        raise ValueError("lse is a contiguous fp32 [n][heads] CUDA tensor")
    batch = _batch(offsets, lengths, page_table, n)
    cache = _cache(k_cache, v_cache, q)
    _check(load().dlrm_kv_attn_fwd(
        ctypes.byref(_heads(q, q)), ctypes.byref(batch), ctypes.byref(cache), d, _TORCH_DTYPES[q.dtype], scale,
        1 if causal else 0, window, max_new, max_len, ctypes.byref(_heads(out, q)), _ptr(lse),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _ptr(err_flag), _stream(stream)),
        "dlrm_kv_attn_fwd")

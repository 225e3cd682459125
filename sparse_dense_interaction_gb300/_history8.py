"""ctypes binding of the event history in 8 bits and of its pages (C ABI:
``include/dlrm_history.h``).

As in :mod:`._history`: argument marshalling only, C names, torch CUDA tensors
of any strides with unit stride in the last dimension.  A cache is a pair of
``float8_e4m3fn`` (or ``uint8``) tensors ``[pages][page_size][heads][d]`` of
codes and a pair of ``uint8`` (or ``float8_e8m0fnu``) tensors ``[pages][blocks
of a page][heads]`` of exponents.  Every tensor is on the current device.
"""
from __future__ import annotations

import struct

import torch

from ._history import _batch, _flag, _heads, _int64, _workspace
from ._native import _TORCH_DTYPES, _check, _ptr, _stream, load

# dlrm_kv_cache8: k, v, k_exp, v_exp, pages, three strides of the codes, three of the exponents, page_size, heads, block
_CACHE8 = struct.Struct("@PPPPqqqqqqqiii4x").pack

_CODES = {torch.float8_e4m3fn, torch.uint8}
_EXPONENTS = {torch.uint8, getattr(torch, "float8_e8m0fnu", torch.uint8)}


def _here(*tensors):
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("every tensor of the call is on the current CUDA device")


def _cache8(k_cache, v_cache, k_exp, v_exp, d):
    strides, exp_strides = k_cache.stride(), k_exp.stride()
    if v_cache.stride() != strides or k_cache.shape != v_cache.shape or v_exp.stride() != exp_strides or (
            k_exp.shape != v_exp.shape):
        raise ValueError("keys and values (codes, exponents) must have one shape and one set of strides")
    pages, page_size, heads, width = k_cache.shape
    page, slot, head, unit = strides
    exp_pages, blocks, exp_heads = k_exp.shape
    if k_cache.dtype not in _CODES or v_cache.dtype is not k_cache.dtype or width != d or (unit != 1 and d > 1):
        raise ValueError("codes are a pair of [pages][page_size][heads][d] float8_e4m3fn tensors, with unit stride in "
                         "the last dimension")
    if k_exp.dtype not in _EXPONENTS or v_exp.dtype is not k_exp.dtype or exp_pages != pages or exp_heads != heads or (
            blocks < 1 or page_size % blocks != 0):
        raise ValueError("exponents are a pair of [pages][blocks][heads] uint8 tensors; the blocks divide a page's slots")
    exp_page, exp_block, exp_head = exp_strides
    return _CACHE8(k_cache.data_ptr(), v_cache.data_ptr(), k_exp.data_ptr(), v_exp.data_ptr(), pages, page, slot, head,
                   exp_page, exp_block, exp_head, page_size, heads, page_size // blocks)


def dlrm_kv8_append(k, v, offsets, lengths, page_table, k_cache, v_cache, k_exp, v_exp, err_flag=None, stream=None):
    """Encodes and stores the new tokens' keys (as they are: normed and turned
    by the caller) and values ``[n][heads][d]`` at the ends of the histories of
    ``lengths`` tokens.

    A block's exponent is the smallest that holds its new tokens, or the one it
    had where it holds older tokens and that is larger; older codes are rounded
    again where it grows."""
    n, _, d = k.shape
    dtype = k.dtype
    _here(k, v, offsets, lengths, page_table, k_cache, v_cache, k_exp, v_exp, err_flag)
    _check(load().dlrm_kv8_append(
        _heads(k, n, d, dtype), _heads(v, n, d, dtype), _batch(offsets, lengths, page_table, n),
        _cache8(k_cache, v_cache, k_exp, v_exp, d), d, _TORCH_DTYPES[dtype], _flag(err_flag), _stream(stream)),
        "dlrm_kv8_append")


def dlrm_kv8_attn_workspace_size(S: int, n: int, q_heads: int, kv_heads: int, d: int, max_new: int,
                                 max_len: int) -> int:
    return load().dlrm_kv8_attn_workspace_size(S, n, q_heads, kv_heads, d, max_new, max_len)


def dlrm_kv8_attn_fwd(q, offsets, lengths, page_table, k_cache, v_cache, k_exp, v_exp, out, scale: float, workspace,
                      max_new: int, max_len: int, causal: bool = True, window: int = 0, lse=None, err_flag=None,
                      stream=None):
    """Attention of the new tokens ``q`` [n][heads][d] (fp32, fp16 or bf16) over
    a cache in 8 bits into ``out`` (same shape and type); the other arguments
    are those of :func:`dlrm_kv_attn_fwd`, with a workspace of
    :func:`dlrm_kv8_attn_workspace_size` bytes."""
    n, heads, d = q.shape
    dtype = q.dtype
    _here(q, offsets, lengths, page_table, k_cache, v_cache, k_exp, v_exp, out, workspace, lse, err_flag)
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (n, heads) or not lse.is_contiguous()):
        raise ValueError("lse is a contiguous fp32 [n][heads] CUDA tensor")
    _check(load().dlrm_kv8_attn_fwd(
        _heads(q, n, d, dtype), _batch(offsets, lengths, page_table, n), _cache8(k_cache, v_cache, k_exp, v_exp, d), d,
        _TORCH_DTYPES[dtype], scale, 1 if causal else 0, window, max_new, max_len, _heads(out, n, d, dtype),
        _ptr(lse), _workspace(workspace), workspace.nbytes, _flag(err_flag), _stream(stream)), "dlrm_kv8_attn_fwd")


def dlrm_kv_reserve(counts, lengths, page_table, page_size: int, ring, state, new_state, offsets, new_lengths,
                    slots=None, positions=None, n=None, err_flag=None, stream=None):
    """Gives out pages and slots for ``counts[s]`` new tokens of each sequence
    that stores ``lengths[s]`` (below 0: it has ended, its pages are given
    back).

    ``ring`` is int32 [pages], of which the entries ``state[0]`` ..
    ``state[1]`` - 1 (modulo pages) are the free pages.  Writes the new pages
    into ``page_table`` (int32 [S][pages]), ``offsets`` (int64 [S + 1]),
    ``new_lengths`` (int64 [S]; may be ``lengths``), ``new_state`` (int64 [2];
    may be ``state``) and, for each new token, ``slots`` and ``positions``
    (int64 [n], both or either; with neither, ``n`` bounds the new tokens)."""
    S = counts.numel()
    rows, width = page_table.shape
    stride, unit = page_table.stride()
    _here(counts, lengths, page_table, ring, state, new_state, offsets, new_lengths, slots, positions, err_flag)
    if page_table.dtype is not torch.int32 or rows != S or (unit != 1 and width > 1):
        raise ValueError("page_table is an int32 [S][pages] CUDA tensor with unit stride in its last dimension")
    if ring.dtype is not torch.int32 or ring.dim() != 1 or not ring.is_contiguous():
        raise ValueError("ring is a contiguous int32 [pages] CUDA tensor")
    if n is None:
        given = slots if slots is not None else positions
        if given is None:
            raise ValueError("n, the most new tokens, is wanted where neither slots nor positions are")
        n = given.numel()
    _check(load().dlrm_kv_reserve(
        _int64(counts, "counts", S), _int64(lengths, "lengths", S), S, n, page_table.data_ptr(), stride, width,
        page_size, ring.data_ptr(), ring.numel(), _int64(state, "state", 2), _int64(new_state, "new_state", 2),
        _int64(offsets, "offsets", S + 1), _int64(new_lengths, "new_lengths", S),
        None if slots is None else _int64(slots, "slots", n),
        None if positions is None else _int64(positions, "positions", n), _flag(err_flag), _stream(stream)),
        "dlrm_kv_reserve")

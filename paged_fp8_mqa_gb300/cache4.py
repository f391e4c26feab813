"""The 4-bit K/V cache: its writer, its reader and the attention over it.

Codes are E2M1, two a byte; keys have a power of two (UE8M0) for each 32 elements, value rows one
float32 scale.  The C-ABI mirrors (``idx_...``) take raw pointers and sizes in the order of
``include/idx.h``, the torch-facing functions take tensors; see ``layer``, whose checks they share.
"""
from __future__ import annotations

import ctypes
import functools

from .layer import (_F, _I, _L, _P, _SIGNATURES, _attend, _c, _check, _code, _elsewhere, _ending, _index,
                    _no_tangents, _on, _rows, _table, _tensor, _tokens)

_SIGNATURES.update({
    "idx_kv_append_fp4": _SIGNATURES["idx_kv_append"],
    "idx_kv_read_fp4": (ctypes.c_int, [_P, _P, _P, _P, _L, _I, _I, _I, _P, _L, _P, _L, _I, _I, _P, _L,
                                       _I, _I, _I, _P, _L, _L, _P, _L, _L, _P]),
    "idx_attention_fp4": _SIGNATURES["idx_attention_fp8"],
})


def idx_kv_append_fp4(*args) -> int:
    return _c("idx_kv_append_fp4")(*args)


def idx_kv_read_fp4(*args) -> int:
    return _c("idx_kv_read_fp4")(*args)


def idx_attention_fp4(*args) -> int:
    return _c("idx_attention_fp4")(*args)


def _cache(k_pool, v_pool, k_scales, v_scales, index):
    """The cache's addresses (k_pool, v_pool, k_scales, v_scales) and sizes (blocks, heads, block_size,
    D)."""
    import torch
    u8 = torch.uint8
    try:  # (the usual case at once; what is wrong with any other is said below)
        shape = blocks, heads, block_size, half = k_pool.shape
        if (k_pool.dtype is u8 and v_pool.dtype is u8 and k_scales.dtype is u8
                and v_scales.dtype is torch.float32 and v_pool.shape == shape
                and k_scales.shape == (blocks, heads, block_size, half // 16)
                and v_scales.shape == (blocks, heads, block_size)
                and k_pool.get_device() == v_pool.get_device() == k_scales.get_device()
                == v_scales.get_device() == index and k_pool.is_contiguous() and v_pool.is_contiguous()
                and k_scales.is_contiguous() and v_scales.is_contiguous()):
            return ((k_pool.data_ptr(), v_pool.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr()),
                    (blocks, heads, block_size, 2 * half))
    except (AttributeError, ValueError):
        pass
    for t, name, dims, dtype in ((k_pool, "k_pool", 4, u8), (v_pool, "v_pool", 4, u8),
                                 (k_scales, "k_scales", 4, u8), (v_scales, "v_scales", 3, torch.float32)):
        _tensor(t, name, dims, dtype, index)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    blocks, heads, block_size, half = k_pool.shape
    if v_pool.shape != k_pool.shape:
        raise ValueError("k_pool and v_pool must both be [blocks, Hkv, block_size, D / 2]")
    rows = (blocks, heads, block_size)
    if k_scales.shape != (*rows, half // 16) or v_scales.shape != rows:
        raise ValueError("k_scales must be [blocks, Hkv, block_size, D / 32], v_scales [blocks, Hkv, "
                         "block_size]")
    return ((k_pool.data_ptr(), v_pool.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr()),
            (*rows, 2 * half))


def kv_append_fp4(k, v, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens, *,
                  token_starts=None, table=None, interleaved: bool = False, rot_offset: int = 0,
                  stream=None):
    """New keys (rotated) and values, [T, Hkv, D] with D = 64 or 128, into the 4-bit cache: pools uint8
    [blocks, Hkv, block_size, D / 2] (E2M1, the even element in the low half of a byte), k_scales uint8
    [blocks, Hkv, block_size, D / 32] (UE8M0: 2^(byte - 127) for each 32 elements), v_scales float32
    [blocks, Hkv, block_size].  The T rows are placed as in ``kv_append``; what a block holds besides
    them stays as it is."""
    import torch
    index = _index(k, "k")
    if index != torch.cuda.current_device():
        return _elsewhere(index, kv_append_fp4, k, v, k_pool, v_pool, k_scales, v_scales, block_tables,
                          seq_lens, token_starts=token_starts, table=table, interleaved=interleaved,
                          rot_offset=rot_offset, stream=stream)
    code, (k_token, k_head, _) = _rows(k, "k", 3, index)
    v_code, (v_token, v_head, _) = _rows(v, "v", 3, index)
    T, H, D = k.shape
    if v_code != code or v.shape != k.shape:
        raise TypeError("k and v must have the same dtype and shape")
    (kp, vp, ks, vs), (blocks, heads, block_size, dim) = _cache(k_pool, v_pool, k_scales, v_scales, index)
    if heads != H or dim != D:
        raise ValueError("the pools must have the heads and the head_dim of k [T, Hkv, D]")
    place = _tokens(block_tables, seq_lens, token_starts, T, index)
    if T and H:
        _check(idx_kv_append_fp4(
            k.data_ptr(), k_token, k_head, v.data_ptr(), v_token, v_head, code, T, H, D,
            *_table(table, index), rot_offset, interleaved, *place, block_size, blocks, kp, vp, ks, vs,
            _on(stream, index)))


def kv_read_fp4(k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens, token_starts=None, *,
                tokens: int, dtype=None, k_out=None, v_out=None, stream=None):
    """What the 4-bit cache holds of the requests' newest tokens, as dense rows: (k, v), [tokens, Hkv, D]
    of dtype (bfloat16 unless given), request b's in rows [token_starts[b], token_starts[b+1]) (int32
    [B + 1]; None: the same number for each).  For an attention among the tokens of a prompt that continues
    what is cached, or a cache of another kind.  Rows that belong to no request, or lie before its first
    token, are zeros in new outputs and stay as they were in given ones."""
    import torch
    index = _index(k_pool, "k_pool")
    if index != torch.cuda.current_device():
        return _elsewhere(index, kv_read_fp4, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens,
                          token_starts, tokens=tokens, dtype=dtype, k_out=k_out, v_out=v_out,
                          stream=stream)
    pools, (blocks, H, block_size, D) = _cache(k_pool, v_pool, k_scales, v_scales, index)
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out are given both or not at all")
    made = []
    if k_out is None:
        dtype = torch.bfloat16 if dtype is None else dtype
        code = _code(dtype)
        if code is None:
            raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
        if tokens < 0:
            raise ValueError("tokens must not be negative")
        made = [torch.empty((tokens, H, D), dtype=dtype, device=k_pool.device) for _ in range(2)]
        k_out, v_out = made
        k_token = v_token = H * D
        k_head = v_head = D
    else:
        code, (k_token, k_head, _) = _rows(k_out, "k_out", 3, index)
        v_code, (v_token, v_head, _) = _rows(v_out, "v_out", 3, index)
        if v_code != code or (dtype is not None and k_out.dtype != dtype):
            raise TypeError("k_out and v_out must have the same dtype, the one asked for")
        if k_out.shape != (tokens, H, D) or v_out.shape != (tokens, H, D):
            raise ValueError("k_out and v_out must be [tokens, Hkv, D]")
        if (tokens > 1 and not (k_token and v_token)) or (H > 1 and not (k_head and v_head)):
            raise ValueError("k_out and v_out must not repeat rows (expanded tensors)")
    starts, lens, stride, batch, next_n, tables, row_stride, width = _tokens(
        block_tables, seq_lens, token_starts, tokens, index)
    if tokens and not batch:
        raise ValueError("tokens of no request")
    if tokens and H and D:
        _check(idx_kv_read_fp4(*pools, blocks, block_size, H, D, starts, tokens, lens, stride, batch,
                               next_n, tables, row_stride, width, bool(made), code,
                               k_out.data_ptr(), k_token, k_head, v_out.data_ptr(), v_token, v_head,
                               _on(stream, index, *made)))
    return k_out, v_out


def attention_fp4(q, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens, *,
                  softmax_scale: float | None = None, candidates=None, ranges=None, out=None,
                  lse=None, workspace=None, num_sms: int = 0, stream=None):
    """``attention_fp8`` over the 4-bit cache (pools and scales as for ``kv_append_fp4``): the same
    queries, extents, candidates, outputs and workspace, and no gradient either.

    It reads half of the bytes, but is not faster everywhere: selected positions (``candidates``) and, with
    head_dim 64, several draft slots take a tenth to a quarter longer than over the 8-bit cache."""
    import torch
    index = _index(q, "q")
    _no_tangents("attention_fp4", q)
    if q.requires_grad and out is None and torch.is_grad_enabled():
        return _ending()(q, "attention_fp4", functools.partial(
            attention_fp4, q, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens,
            softmax_scale=softmax_scale, candidates=candidates, ranges=ranges, lse=lse,
            workspace=workspace, num_sms=num_sms, stream=stream))
    if index != torch.cuda.current_device():
        return _elsewhere(index, attention_fp4, q, k_pool, v_pool, k_scales, v_scales, block_tables,
                          seq_lens, softmax_scale=softmax_scale, candidates=candidates,
                          ranges=ranges, out=out, lse=lse, workspace=workspace, num_sms=num_sms,
                          stream=stream)
    pools, sizes = _cache(k_pool, v_pool, k_scales, v_scales, index)
    return _attend(idx_attention_fp4, index, q, pools, sizes, block_tables, seq_lens, softmax_scale,
                   candidates, ranges, out, lse, workspace, num_sms, stream)

"""The operators around the indexer: rotary positions, the writers of the two 8-bit pools and the
attention over the K/V pool.

Like the rest of the binding it only marshals: the C-ABI mirrors (``idx_...``) take raw pointers
and sizes in the order of ``include/idx.h``, the torch-facing functions take tensors.  Tensors that
a call allocates (outputs, workspace) belong to PyTorch's caching allocator; they are recorded on
``stream`` when it is not the current one.
"""
from __future__ import annotations

import ctypes
import functools

IDX_ROTARY_NONE = 0
IDX_ROTARY_LINEAR = 1
IDX_ROTARY_NTK = 2
IDX_ROTARY_YARN = 3
IDX_ROTARY_MAX_DIM = 1024

_SCALINGS = {"none": IDX_ROTARY_NONE, "linear": IDX_ROTARY_LINEAR, "ntk": IDX_ROTARY_NTK,
             "yarn": IDX_ROTARY_YARN}

_P, _I, _L, _F, _D = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                      ctypes.c_double)
_SIGNATURES = {
    "idx_rotary_frequencies": (ctypes.c_int, [_I, _D, _I, _D, _D, _D, _D, _P, _P]),
    "idx_rotary_table": (ctypes.c_int, [_P, _D, _I, _I, _P, _P]),
    "idx_rotary": (ctypes.c_int, [_P, _L, _L, _P, _L, _I, _I, _I, _P, _I, _I, _I, _I, _I, _P, _L,
                                  _L, _P]),
    "idx_index_prepare": (ctypes.c_int, [_P, _L, _P, _L, _L, _P, _L, _I, _L, _I, _I, _P, _I, _I,
                                         _I, _I, _P, _P, _L, _I, _I, _P, _L, _I, _I, _L, _P, _P,
                                         _P, _P]),
    "idx_kv_append": (ctypes.c_int, [_P, _L, _L, _P, _L, _L, _I, _L, _I, _I, _P, _I, _I, _I, _I,
                                     _P, _P, _L, _I, _I, _P, _L, _I, _I, _L, _P, _P, _P, _P, _P]),
    "idx_attention_workspace_bytes": (ctypes.c_int64, [_I, _I, _I, _I, _I, _I]),
    "idx_attention_fp8": (ctypes.c_int, [_P, _L, _L, _L, _I, _P, _P, _P, _P, _L, _I, _P, _L, _I,
                                         _P, _L, _I, _I, _I, _I, _I, _F, _P, _I, _P, _I, _P, _P,
                                         _P, _L, _P]),
}
_functions: dict = {}


def _c(name):
    f = _functions.get(name)
    if f is None:
        from . import lib
        f = getattr(lib(), name)
        f.restype, f.argtypes = _SIGNATURES[name]
        _functions[name] = f
    return f


# ---- C-ABI mirrors (raw pointers / ints) -------------------------------------------------------

def idx_rotary_frequencies(*args) -> int:
    return _c("idx_rotary_frequencies")(*args)


def idx_rotary_table(*args) -> int:
    return _c("idx_rotary_table")(*args)


def idx_rotary(*args) -> int:
    return _c("idx_rotary")(*args)


def idx_index_prepare(*args) -> int:
    return _c("idx_index_prepare")(*args)


def idx_kv_append(*args) -> int:
    return _c("idx_kv_append")(*args)


def idx_attention_workspace_bytes(*args) -> int:
    return int(_c("idx_attention_workspace_bytes")(*args))


def idx_attention_fp8(*args) -> int:
    return _c("idx_attention_fp8")(*args)


# ---- torch-facing marshalling ------------------------------------------------------------------

_codes: dict = {}
_sizes: dict = {}


def _code(dtype):
    """The IDX_DTYPE_* code of float32, float16 or bfloat16, or None."""
    if not _codes:
        import torch
        from . import IDX_DTYPE_BF16, IDX_DTYPE_F16, IDX_DTYPE_F32
        _codes.update({torch.float32: IDX_DTYPE_F32, torch.float16: IDX_DTYPE_F16,
                       torch.bfloat16: IDX_DTYPE_BF16})
    return _codes.get(dtype)


def _check(status: int) -> None:
    if status:
        from . import IdxError, idx_last_error
        raise IdxError(status, idx_last_error())


def _index(t, name):
    """The device index of a CUDA tensor."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _elsewhere(index, f, *args, **more):
    """f again with device `index`, its tensors', current: the launch, the SM count and the workspace's
    size are then that device's.  (Each call asks for itself whether it has to: a wrapper around it
    costs a microsecond.)"""
    import torch
    with torch.cuda.device(index):
        return f(*args, **more)


def _tensor(t, name, dims, dtype, index):
    """A CUDA tensor of dtype on device `index` with `dims` dimensions.  (One test for the usual
    case: a call's checks are a good part of its time on the host.)"""
    try:
        if t.dtype is dtype and t.get_device() == index and t.dim() == dims:
            return
    except AttributeError:
        pass
    if _index(t, name) != index:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not on cuda:{index}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got {t.dim()}")


def _rows(t, name, dims, index):
    """Rows of float32, float16 or bfloat16 elements with unit element stride: their dtype code and
    strides."""
    if _index(t, name) != index:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not on cuda:{index}")
    code = _code(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    strides = t.stride()
    if len(strides) != dims:
        raise ValueError(f"{name} must have {dims} dims, got {len(strides)}")
    if strides[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} rows must be contiguous")
    return code, strides


def _pool8(t, name, dims, index):
    """e4m3 values (or their uint8 view), contiguous: their address."""
    import torch
    raw = getattr(t, "dtype", None) is torch.uint8
    _tensor(t, name, dims, torch.uint8 if raw else torch.float8_e4m3fn, index)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _scales(t, name, shape, index):
    """A pool's float32 scales [blocks, Hkv]: their address."""
    import torch
    _tensor(t, name, 2, torch.float32, index)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [blocks, Hkv]")
    return t.data_ptr()


def _on(stream, index, *allocated):
    """The raw stream to launch on; tensors allocated for another stream's work are recorded."""
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream != torch.cuda.current_stream(index):
        for t in allocated:
            t.record_stream(stream)
    return stream.cuda_stream


def _table(table, index):
    """(pointer, max_positions, rot_dim) of a rotary table, or of none."""
    import torch
    if table is None:
        return None, 0, 0
    _tensor(table, "table", 3, torch.float32, index)
    most, half, two = table.shape
    if two != 2 or not table.is_contiguous():
        raise ValueError("table must be contiguous [max_positions, rot_dim / 2, 2]")
    return table.data_ptr(), most, 2 * half


def _requests(block_tables, seq_lens, batch, index):
    """The arguments of a batch's pages: (block_tables, row stride, width, seq_lens, stride)."""
    import torch
    _tensor(block_tables, "block_tables", 2, torch.int32, index)
    _tensor(seq_lens, "seq_lens", 1, torch.int32, index)
    rows, width = block_tables.shape
    if batch is None:
        batch = rows
    if rows != batch or seq_lens.shape[0] != batch:
        raise ValueError("block_tables and seq_lens must have a row for each request")
    row_stride, unit = block_tables.stride()
    if width > 1 and unit != 1:
        raise ValueError("block_tables rows must be contiguous (stride(1) == 1)")
    len_stride, = seq_lens.stride()
    if batch < 2:  # (the stride of a single row means nothing)
        row_stride, len_stride = width, 1
    elif row_stride < width or len_stride < 1:
        raise ValueError("block_tables and seq_lens must not repeat rows (expanded tensors)")
    return block_tables.data_ptr(), row_stride, width, seq_lens.data_ptr(), len_stride


def _tokens(block_tables, seq_lens, token_starts, rows, index):
    """The arguments that place new tokens: (starts, seq_lens, stride, batch, next_n, tables, row
    stride, width)."""
    import torch
    tables, row_stride, width, lens, stride = _requests(block_tables, seq_lens, None, index)
    batch = seq_lens.shape[0]
    starts, next_n = None, 0
    if token_starts is not None:
        _tensor(token_starts, "token_starts", 1, torch.int32, index)
        if token_starts.shape[0] != batch + 1 or not token_starts.is_contiguous():
            raise ValueError("token_starts must be contiguous, one more than the requests")
        starts = token_starts.data_ptr()
    elif batch:
        next_n = rows // batch
        if next_n * batch != rows:
            raise ValueError("without token_starts every request has the same number of tokens")
    return starts, lens, stride, batch, next_n, tables, row_stride, width


def rotary_table(max_positions: int, rot_dim: int, *, base: float = 10000.0, scaling: str = "none",
                 factor: float = 1.0, original_positions: float = 0.0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, device=None, stream=None):
    """The cosine and sine of every position's angles, float32 [max_positions, rot_dim / 2, 2],
    computed in 64 bits.  scaling: "none", "linear" (angles divided by factor), "ntk" (the base
    grows) or "yarn" (by parts: pairs that turn at least beta_fast times over original_positions
    are left alone, those that turn at most beta_slow times are divided by factor, and the cosines
    and sines are multiplied by 0.1 ln(factor) + 1).  Built once and kept by the caller."""
    import torch
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    freq = (ctypes.c_double * max(1, rot_dim // 2))()
    magnitude = ctypes.c_double()
    _check(idx_rotary_frequencies(rot_dim, base, _SCALINGS[scaling], factor, original_positions,
                                  beta_fast, beta_slow, freq, ctypes.byref(magnitude)))
    device = torch.device("cuda" if device is None else device)
    with torch.cuda.device(device):
        table = torch.empty(max_positions, rot_dim // 2, 2, dtype=torch.float32, device=device)
        _check(idx_rotary_table(freq, magnitude.value, max_positions, rot_dim, table.data_ptr(),
                                _on(stream, table.get_device(), table)))
    return table


@functools.cache
def _recorded_rotary():
    """rotary as a step that autograd records: its backward is rotary the other way."""
    import torch

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, positions, table, interleaved, rot_offset, inverse, stream):
            ctx.save_for_backward(positions, table)
            ctx.how = dict(interleaved=interleaved, rot_offset=rot_offset, inverse=not inverse)
            return rotary(x, positions, table, interleaved=interleaved, rot_offset=rot_offset,
                          inverse=inverse, stream=stream)

        @staticmethod
        def backward(ctx, grad):
            positions, table = ctx.saved_tensors
            if grad.shape[-1] > 1 and grad.stride(-1) != 1:  # (of a sum: one element, expanded)
                grad = grad.contiguous()
            return (rotary(grad, positions, table, **ctx.how), *[None] * 6)

    return Rotary.apply


def rotary(x, positions, table, *, interleaved: bool = False, rot_offset: int = 0,
           inverse: bool = False, out=None, stream=None):
    """Rotary positions: x [T, H, D] (float32, float16 or bfloat16; any token and head strides) at
    positions (int32 [T]), elements [rot_offset, rot_offset + rot_dim) of each head turned by the
    angles of ``table`` (see ``rotary_table``), in halves or in interleaved pairs.  ``out=x``
    rotates in place.  ``inverse`` turns by the negative angles: the gradient with respect to x (and
    the way back, where the table's magnitude is 1, as it is but for "yarn").  Autograd records the
    call where x requires a gradient; with ``out`` nothing is recorded."""
    import torch
    index = _index(x, "x")
    if x.requires_grad and out is None and torch.is_grad_enabled():
        return _recorded_rotary()(x, positions, table, interleaved, rot_offset, inverse, stream)
    if index != torch.cuda.current_device():
        return _elsewhere(index, rotary, x, positions, table, interleaved=interleaved,
                          rot_offset=rot_offset, inverse=inverse, out=out, stream=stream)
    code, (x_token, x_head, _) = _rows(x, "x", 3, index)
    _tensor(positions, "positions", 1, torch.int32, index)
    T, H, D = x.shape
    if positions.shape[0] != T or not positions.is_contiguous():
        raise ValueError("positions must be contiguous, one for each token of x")
    tab, most, rot = _table(table, index)
    if tab is None:
        raise TypeError("table must be a CUDA tensor")
    made = ()
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
        made = (out,)
        o_token, o_head = H * D, D
    else:
        _tensor(out, "out", 3, x.dtype, index)
        if out.shape != x.shape or (D > 1 and out.stride(2) != 1):
            raise ValueError("out must have the shape of x and contiguous rows")
        o_token, o_head, _ = out.stride()
    if not (T and H and D):
        return out
    _check(idx_rotary(x.data_ptr(), x_token, x_head, positions.data_ptr(), T, H, D, code, tab, most,
                      rot, rot_offset, interleaved, inverse, out.data_ptr(), o_token, o_head,
                      _on(stream, index, *made)))
    return out


def index_prepare(k, kv_fused, block_tables, seq_lens, *, token_starts=None, q=None, weights=None,
                  table=None, interleaved: bool = False, rot_offset: int = 0, q_out=None,
                  weights_out=None, stream=None):
    """The inputs of ``logits_fp8`` from a layer's index keys and queries.

    k [T, D] (D = 64, 128 or 192) is rotated, quantised to e4m3 with a float32 scale for each row
    and written to the requests' pages of ``kv_fused``; the T rows are the requests' newest tokens,
    the same number for each, or rows [token_starts[b], token_starts[b+1]) (int32 [B + 1]);
    seq_lens counts them already.  q [T, H, D] with weights [T, H] float32, if given, is rotated
    and quantised likewise, its scales folded into the weights: returns (q e4m3 [T, H, D],
    weights float32 [T, H]), which ``logits_fp8`` takes (q viewed as [B, next_n, H, D])."""
    import torch
    index = _index(k, "k")
    if index != torch.cuda.current_device():
        return _elsewhere(index, index_prepare, k, kv_fused, block_tables, seq_lens,
                          token_starts=token_starts, q=q, weights=weights, table=table,
                          interleaved=interleaved, rot_offset=rot_offset, q_out=q_out,
                          weights_out=weights_out, stream=stream)
    code, (k_token, _) = _rows(k, "k", 2, index)
    T, D = k.shape
    if _index(kv_fused, "kv_fused") != index or kv_fused.dtype is not torch.uint8:
        raise TypeError("kv_fused must be a uint8 tensor on the device of k")
    blocks = kv_fused.shape[0] if kv_fused.dim() else 0
    if blocks == 0 or not kv_fused.is_contiguous():
        raise ValueError("kv_fused must be contiguous with a leading dim of blocks")
    block_size, rest = divmod(kv_fused.numel() // blocks, D + 4)
    if rest:
        raise ValueError(f"kv_fused blocks must be block_size * (D + 4) bytes, D = {D}")
    H, made = 0, []
    q_args, q_to, w_to = (None, 0, 0, None, 0), None, None
    if q is not None:
        q_code, (q_token, q_head, _) = _rows(q, "q", 3, index)
        if q_code != code:
            raise TypeError("q and k must have the same dtype")
        _tensor(weights, "weights", 2, torch.float32, index)
        H = q.shape[1]
        w_token, w_head = weights.stride()
        if q.shape != (T, H, D) or weights.shape != (T, H):
            raise ValueError("q must be [T, H, D] and weights [T, H] for k [T, D]")
        if H > 1 and w_head != 1:
            raise ValueError("weights rows must be contiguous")
        if q_out is None:
            q_out = torch.empty((T, H, D), dtype=torch.float8_e4m3fn, device=k.device)
            made.append(q_out)
        if weights_out is None:
            weights_out = torch.empty((T, H), dtype=torch.float32, device=k.device)
            made.append(weights_out)
        q_to = _pool8(q_out, "q_out", 3, index)
        _tensor(weights_out, "weights_out", 2, torch.float32, index)
        if q_out.shape != q.shape or weights_out.shape != weights.shape \
                or not weights_out.is_contiguous():
            raise ValueError("q_out and weights_out must be contiguous with the shapes of q and "
                             "weights")
        if H:
            w_to = weights_out.data_ptr()
            q_args = (q.data_ptr(), q_token, q_head, weights.data_ptr(), w_token)
        else:  # the keys alone
            q_to = None
    place = _tokens(block_tables, seq_lens, token_starts, T, index)
    if T:
        _check(idx_index_prepare(
            k.data_ptr(), k_token, *q_args, code, T, H, D, *_table(table, index), rot_offset,
            interleaved, *place, block_size, blocks, kv_fused.data_ptr(), q_to, w_to,
            _on(stream, index, *made)))
    return None if q is None else (q_out, weights_out)


def kv_append(k, v, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens, *,
              token_starts=None, table=None, interleaved: bool = False, rot_offset: int = 0,
              stream=None):
    """New keys (rotated) and values, [T, Hkv, D] with D = 64 or 128, into the 8-bit cache: pools
    e4m3 [blocks, Hkv, block_size, D], scales float32 [blocks, Hkv] (powers of two).  The T rows
    are placed as in ``index_prepare``.  A block that already holds tokens keeps its scale while
    the new ones fit it; otherwise the scale grows and what it holds is rescaled."""
    import torch
    index = _index(k, "k")
    if index != torch.cuda.current_device():
        return _elsewhere(index, kv_append, k, v, k_pool, v_pool, k_scales, v_scales, block_tables,
                          seq_lens, token_starts=token_starts, table=table, interleaved=interleaved,
                          rot_offset=rot_offset, stream=stream)
    code, (k_token, k_head, _) = _rows(k, "k", 3, index)
    v_code, (v_token, v_head, _) = _rows(v, "v", 3, index)
    shape = T, H, D = k.shape
    if v_code != code or v.shape != shape:
        raise TypeError("k and v must have the same dtype and shape")
    pools = _pool8(k_pool, "k_pool", 4, index), _pool8(v_pool, "v_pool", 4, index)
    blocks, heads, block_size, dim = k_pool.shape
    if heads != H or dim != D or v_pool.shape != k_pool.shape:
        raise ValueError("k_pool and v_pool must be [blocks, Hkv, block_size, D] for k [T, Hkv, D]")
    scales = (_scales(k_scales, "k_scales", (blocks, H), index),
              _scales(v_scales, "v_scales", (blocks, H), index))
    place = _tokens(block_tables, seq_lens, token_starts, T, index)
    if T and H:
        _check(idx_kv_append(
            k.data_ptr(), k_token, k_head, v.data_ptr(), v_token, v_head, code, T, H, D,
            *_table(table, index), rot_offset, interleaved, *place, block_size, blocks, *pools,
            *scales, _on(stream, index)))


def attention_fp8(q, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens, *,
                  softmax_scale: float | None = None, candidates=None, ranges=None, out=None,
                  lse=None, workspace=None, num_sms: int = 0, stream=None):
    """Attention over the 8-bit K/V cache: q [B, next_n, H, D] (float16 or bfloat16; strides that
    are multiples of 8), pools and scales as for ``kv_append``, H a multiple of Hkv; row (b, t)
    sees positions 0 .. seq_lens[b] - next_n + t.  With ``candidates`` (int32 [B*next_n, slots, 2])
    and ``ranges`` (int32 [2, B*next_n]) as the select leaves them, each row sees only the
    positions stored in its slot range.  Rows that see nothing give zeros.  softmax_scale defaults
    to D ** -0.5; weights are held to 2^-10 of themselves (float16 queries: 2^-14), sums in float32;
    ``lse`` (float32 [B, next_n, H]) receives the log-sums; ``workspace`` (uint8, at
    least idx_attention_workspace_bytes) is allocated if not given.  Returns out, contiguous
    [B, next_n, H, D] in q's dtype."""
    import torch
    index = _index(q, "q")
    if index != torch.cuda.current_device():
        return _elsewhere(index, attention_fp8, q, k_pool, v_pool, k_scales, v_scales, block_tables,
                          seq_lens, softmax_scale=softmax_scale, candidates=candidates,
                          ranges=ranges, out=out, lse=lse, workspace=workspace, num_sms=num_sms,
                          stream=stream)
    dtype = q.dtype
    code = _code(dtype)
    if code is None or dtype is torch.float32:
        raise TypeError(f"q must be float16 or bfloat16, got {dtype}")
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"q must have 4 dims, got {len(shape)}")
    B, n, H, D = shape
    q_batch, q_token, q_head, q_unit = q.stride()
    if q_unit != 1 and D > 1:
        raise ValueError("q rows must be contiguous")
    pools = _pool8(k_pool, "k_pool", 4, index), _pool8(v_pool, "v_pool", 4, index)
    blocks, kv_heads, block_size, dim = k_pool.shape
    if dim != D or v_pool.shape != k_pool.shape:
        raise ValueError("k_pool and v_pool must be [blocks, Hkv, block_size, D] for q's D")
    scales = (_scales(k_scales, "k_scales", (blocks, kv_heads), index),
              _scales(v_scales, "v_scales", (blocks, kv_heads), index))
    pages = _requests(block_tables, seq_lens, B, index)
    cand, slots, cand_ranges = None, 0, None
    if candidates is not None:
        _tensor(candidates, "candidates", 3, torch.int32, index)
        if ranges is None:
            raise ValueError("ranges is required with candidates")
        _tensor(ranges, "ranges", 2, torch.int32, index)
        rows, slots, pair = candidates.shape
        if rows != B * n or pair != 2 or not candidates.is_contiguous():
            raise ValueError("candidates must be contiguous [B * next_n, slots, 2]")
        if ranges.shape != (2, rows) or not ranges.is_contiguous():
            raise ValueError("ranges must be contiguous [2, B * next_n]")
        cand, cand_ranges = candidates.data_ptr(), ranges.data_ptr()
    made = []
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
        made.append(out)
    else:
        _tensor(out, "out", 4, dtype, index)
        if out.shape != shape or not out.is_contiguous():
            raise ValueError("out must be contiguous with the shape of q")
    lse_to = None
    if lse is not None:
        _tensor(lse, "lse", 3, torch.float32, index)
        if lse.shape != shape[:3] or not lse.is_contiguous():
            raise ValueError("lse must be contiguous [B, next_n, H]")
        lse_to = lse.data_ptr()
    if not (B and n and H and D):
        return out
    if workspace is None:
        sizes = (index, B, n, H, kv_heads, D, num_sms)
        need = _sizes.get(sizes)
        if need is None:
            need = idx_attention_workspace_bytes(*sizes[1:])
            if need >= 0 and len(_sizes) < 4096:  # (-1: the call below says what is wrong)
                _sizes[sizes] = need
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
        made.append(workspace)
    else:
        _tensor(workspace, "workspace", 1, torch.uint8, index)
        need = workspace.shape[0]
    _check(idx_attention_fp8(
        q.data_ptr(), q_batch, q_token, q_head, code, *pools, *scales, blocks, block_size, *pages,
        B, n, H, kv_heads, D, D ** -0.5 if softmax_scale is None else softmax_scale, cand, slots,
        cand_ranges, num_sms, out.data_ptr(), lse_to, workspace.data_ptr(), need,
        _on(stream, index, *made)))
    return out

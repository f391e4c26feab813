"""Heads rotated by several axes, and queries and keys normalised and rotated at once.

The C-ABI mirrors (``idx_...``) take raw pointers and sizes in the order of ``include/idx.h``, the
torch-facing functions take tensors; see ``layer``, whose checks they share.
"""
from __future__ import annotations

import ctypes
import functools

from .layer import (_F, _I, _L, _P, _SIGNATURES, _c, _check, _code, _elsewhere, _index, _no_tangents, _on, _rows,
                    _table, _tensor)

IDX_ROTARY_MAX_AXES = 4
IDX_NORM_MAX_DIM = 1024

_ROWS = [_P, _L, _L]
_TURN = [_P, _L, _P, _I, _P, _I, _I, _I, _I]  # positions, axes, table, pairs
_NORM = [*_ROWS, _I, *_ROWS, _I, _I, _L, _I, _P, _P, _I, _F, *_TURN]
_SIGNATURES.update({
    "idx_rotary_axes": (ctypes.c_int, [*_ROWS, _P, _L, _P, _I, _L, _I, _I, _I, _P, _I, _I, _I, _I, _I,
                                       *_ROWS, _P]),
    "idx_norm_rotary": (ctypes.c_int, [*_NORM, *_ROWS, *_ROWS, _P]),
    "idx_norm_rotary_workspace_bytes": (ctypes.c_int64, [_I]),
    "idx_norm_rotary_backward": (ctypes.c_int, [*_NORM, *_ROWS, *_ROWS, _P, _P, _P, _P, _P, _L, _P]),
})


def idx_rotary_axes(*args) -> int:
    return _c("idx_rotary_axes")(*args)


def idx_norm_rotary(*args) -> int:
    return _c("idx_norm_rotary")(*args)


def idx_norm_rotary_workspace_bytes(*args) -> int:
    return int(_c("idx_norm_rotary_workspace_bytes")(*args))


def idx_norm_rotary_backward(*args) -> int:
    return _c("idx_norm_rotary_backward")(*args)


def rotary_axes(sections, *, in_turn: bool = False):
    """The axis of each pair for ``axes=``, from the number of pairs of each axis: one section after
    the other, or, ``in_turn``, one pair of each axis after the other while it has some left."""
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= IDX_ROTARY_MAX_AXES or min(left) < 0:
        raise ValueError(f"sections must be 1 to {IDX_ROTARY_MAX_AXES} numbers of pairs")
    if not in_turn:
        return tuple(a for a, n in enumerate(left) for _ in range(n))
    return tuple(a for i in range(max(left)) for a, n in enumerate(left) if i < n)


@functools.lru_cache(maxsize=256)
def _axis_bytes(axes, count, pairs):
    """The axes of all pairs as the C entry takes them (host memory)."""
    if len(axes) != pairs:
        raise ValueError(f"axes must name an axis for each of the {pairs} pairs, got {len(axes)}")
    if any(not isinstance(a, int) or not 0 <= a < count for a in axes):
        raise ValueError(f"axes must be whole numbers below the {count} axes of positions")
    return (ctypes.c_uint8 * pairs)(*axes)


def _turn(positions, axes, rot, T, index):
    """The arguments (positions, axis stride, pair_axis, axes) of a rotation."""
    import torch
    if axes is None:
        _tensor(positions, "positions", 1, torch.int32, index)
        if positions.shape[0] != T or not positions.is_contiguous():
            raise ValueError("positions must be contiguous, one for each token")
        return positions.data_ptr(), 0, None, 1
    _tensor(positions, "positions", 2, torch.int32, index)
    count = positions.shape[0]
    if positions.shape[1] != T or not 1 <= count <= IDX_ROTARY_MAX_AXES:
        raise ValueError(f"positions must be [axes, T] with 1 to {IDX_ROTARY_MAX_AXES} axes")
    axis_stride, unit = positions.stride()
    if T > 1 and unit != 1:
        raise ValueError("positions of an axis must be contiguous")
    pair_axis = _axis_bytes(axes, count, rot // 2)
    return positions.data_ptr(), axis_stride, pair_axis, count


def _like(out, x, name, index, made):
    """The result for x: ``out`` if given, else a new one; and its strides."""
    import torch
    if out is None:
        shape = x.shape
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        made.append(out)
        return out, shape[1] * shape[2], shape[2]
    _tensor(out, name, 3, x.dtype, index)
    token, head, unit = out.stride()
    if out.shape != x.shape or (x.shape[2] > 1 and unit != 1):
        raise ValueError(f"{name} must have its input's shape and contiguous rows")
    if (x.shape[0] > 1 and token == 0) or (x.shape[1] > 1 and head == 0):
        raise ValueError(f"{name} must not repeat rows (an expanded tensor)")
    return out, token, head


def rotary_by_axes(x, positions, table, axes, interleaved, rot_offset, inverse, out, stream):
    """``rotary`` with ``axes`` (on x's device, which is the current one)."""
    index = _index(x, "x")
    code, (x_token, x_head, _) = _rows(x, "x", 3, index)
    T, H, D = x.shape
    tab, most, rot = _table(table, index)
    if tab is None:
        raise TypeError("table must be a CUDA tensor")
    place, axis_stride, pair_axis, count = _turn(positions, axes, rot, T, index)
    made = []
    out, o_token, o_head = _like(out, x, "out", index, made)
    if not (T and H and D):
        return out
    _check(idx_rotary_axes(x.data_ptr(), x_token, x_head, place, axis_stride, pair_axis, count, T, H, D,
                           code, tab, most, rot, rot_offset, interleaved, inverse, out.data_ptr(),
                           o_token, o_head, _on(stream, index, *made)))
    return out


def _weight(w, name, code, D, index):
    """A weight's address and dtype code."""
    if w is None:
        return None, None
    if _index(w, name) != index:
        raise ValueError(f"{name} is on cuda:{w.get_device()}, not on cuda:{index}")
    w_code = _code(w.dtype)
    if w_code not in (code, 0):  # (IDX_DTYPE_F32)
        raise TypeError(f"{name} must have the dtype of q and k, or float32")
    if w.shape != (D,) or not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{D}]")
    return w.data_ptr(), w_code


def _norm_args(q, k, q_weight, k_weight, positions, table, eps, axes, interleaved, rot_offset, index):
    """The arguments that the forward and the backward entry share."""
    code, (q_token, q_head, _) = _rows(q, "q", 3, index)
    T, H, D = q.shape
    k_at, k_token, k_head, k_heads = None, 0, 0, 0
    if k is not None:
        k_code, (k_token, k_head, _) = _rows(k, "k", 3, index)
        k_T, k_heads, k_D = k.shape
        if k_code != code or k_T != T or k_D != D:
            raise TypeError("q and k must have the same dtype, tokens and head_dim")
        k_at = k.data_ptr() if k_heads else None
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    if q_weight is not None and k_weight is not None and q_weight.dtype is k_weight.dtype \
            and q_weight.shape == k_weight.shape == (D,) and q_weight.get_device() == index \
            and k_weight.get_device() == index and q_weight.is_contiguous() and k_weight.is_contiguous() \
            and _code(q_weight.dtype) in (code, 0):
        qw, kw, w_code = q_weight.data_ptr(), k_weight.data_ptr(), _code(q_weight.dtype)
    else:
        qw, qw_code = _weight(q_weight, "q_weight", code, D, index)
        kw, kw_code = _weight(k_weight, "k_weight", code, D, index)
        if qw_code is not None and kw_code is not None and qw_code != kw_code:
            raise TypeError("q_weight and k_weight must have the same dtype")
        w_code = qw_code if qw_code is not None else kw_code if kw_code is not None else code
    if table is not None:
        tab, most, rot = _table(table, index)
        at, axis_stride, pair_axis, count = _turn(positions, axes, rot, T, index)
        return (q.data_ptr(), q_token, q_head, H, k_at, k_token, k_head, k_heads, code, T, D, qw, kw,
                w_code, eps, at, axis_stride, pair_axis, count, tab, most, rot, rot_offset, interleaved)
    if positions is not None or axes is not None:
        raise ValueError("positions and axes need a table")
    return (q.data_ptr(), q_token, q_head, H, k_at, k_token, k_head, k_heads, code, T, D, qw, kw, w_code,
            eps, None, 0, None, 1, None, 0, 0, rot_offset, interleaved)


def _forward(index, args, q, k, q_out, k_out, stream):
    """The call with the arguments that _norm_args made."""
    made = []
    q_to, q_token, q_head = _like(q_out, q, "q_out", index, made)
    k_to, k_at, k_token, k_head = None, None, 0, 0
    if k is not None:
        k_to, k_token, k_head = _like(k_out, k, "k_out", index, made)
        k_at = k_to.data_ptr() if args[7] else None
    if args[9] and args[10] and args[3] + args[7]:
        # (Without query heads there is nothing at q: any address will do.)
        q_at = q_to.data_ptr() if args[3] else k_at
        if not args[3]:
            args = (k_at, *args[1:])
        _check(idx_norm_rotary(*args, q_at, q_token, q_head, k_at, k_token, k_head,
                               _on(stream, index, *made)))
    return q_to, k_to


def _backward(q, k, q_weight, k_weight, positions, table, eps, axes, interleaved, rot_offset, q_grad,
              k_grad, args=None):
    """(dq, dk, dq_weight, dk_weight) from the outputs' gradients.  args: those of the forward call, if
    the tensors are still the ones that it had."""
    import torch
    index = _index(q, "q")
    if index != torch.cuda.current_device():
        return _elsewhere(index, _backward, q, k, q_weight, k_weight, positions, table, eps, axes,
                          interleaved, rot_offset, q_grad, k_grad, args)
    if args is None or args[0] != q.data_ptr():
        args = _norm_args(q, k, q_weight, k_weight, positions, table, eps, axes, interleaved, rot_offset,
                          index)

    def rows(g, x):
        if g.dtype != x.dtype:
            g = g.to(x.dtype)
        if g.shape[2] > 1 and g.stride(2) != 1:  # (of a sum: one element, expanded)
            g = g.contiguous()
        return g

    empty, dtype, device = torch.empty, q.dtype, q.device
    T, D = args[9], args[10]
    dq = empty(q.shape, dtype=dtype, device=device)
    dk = None if k is None else empty(k.shape, dtype=dtype, device=device)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    if not T:  # (sums over nothing)
        return dq, dk, *(None if w is None else w.zero_() for w in (dqw, dkw))
    q_grad = rows(q_grad, q)
    qg_token, qg_head, _ = q_grad.stride()
    kg, kg_token, kg_head, dk_at = None, 0, 0, None
    if k is not None:
        k_grad = rows(k_grad, k)
        kg_token, kg_head, _ = k_grad.stride()
        kg, dk_at = k_grad.data_ptr(), dk.data_ptr()
    need = _workspaces.get((index, D))
    if need is None:
        need = idx_norm_rotary_workspace_bytes(D)
        if need > 0:
            _workspaces[index, D] = need
    workspace = empty(max(need, 1), dtype=torch.uint8, device=device)
    _check(idx_norm_rotary_backward(
        *args, q_grad.data_ptr(), qg_token, qg_head, kg, kg_token, kg_head, dq.data_ptr(), dk_at,
        None if dqw is None else dqw.data_ptr(), None if dkw is None else dkw.data_ptr(),
        workspace.data_ptr(), need, _on(None, index)))
    return dq, dk, dqw, dkw


_workspaces: dict = {}  # sizes, by device and head_dim


@functools.cache
def _recorded():
    """norm_rotary as a step that autograd records."""
    import torch
    from torch.autograd.function import once_differentiable

    class NormRotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_weight, k_weight, positions, table, eps, axes, interleaved, rot_offset,
                    stream):
            index = q.get_device()
            args = _norm_args(q, k, q_weight, k_weight, positions, table, eps, axes, interleaved,
                              rot_offset, index)
            ctx.save_for_backward(q, k, q_weight, k_weight, positions, table)
            ctx.how = eps, axes, interleaved, rot_offset
            ctx.args = args
            ctx.places = None if positions is None else positions.stride()
            return _forward(index, args, q, k, None, None, stream)

        @staticmethod
        @once_differentiable
        def backward(ctx, q_grad, k_grad):
            saved = ctx.saved_tensors
            # (Hooks on what is saved may have put other tensors in their place.)
            a = ctx.args
            q, k, q_weight, k_weight, positions, table = saved
            at = [None if t is None else t.data_ptr() for t in saved]
            same = at == [a[0], a[4], a[11], a[12], a[15], a[19]] and q.stride()[:2] == a[1:3] \
                and (k is None or k.stride()[:2] == a[5:7]) \
                and (positions is None or positions.stride() == ctx.places) \
                and all(t is None or t.is_contiguous() for t in (q_weight, k_weight, table))
            return (*_backward(*saved, *ctx.how, q_grad, k_grad, a if same else None), *[None] * 7)

    return NormRotary.apply


def norm_rotary(q, k, q_weight=None, k_weight=None, positions=None, table=None, *, eps: float = 1e-6,
                axes=None, interleaved: bool = False, rot_offset: int = 0, q_out=None, k_out=None,
                stream=None):
    """Every head of q [T, H, D] and of k [T, Hkv, D] (float32, float16 or bfloat16; any token and head
    strides, so views of one projection do) over its root mean square, times its weight, and rotated as by
    ``rotary``: R(x / sqrt(mean(x^2) + eps) * weight), one launch, float32 within, one rounding.

    The weights [D] (their dtype or float32; None: ones) belong to all heads of q and of k.  k may be
    None.  Without a table nothing is rotated; with ``axes`` (see ``rotary_axes``) positions are
    int32 [axes, T].  ``q_out=q`` and ``k_out=k`` work in place.  Returns (q, k) normalised.

    Autograd records the call where q, k or a weight requires a gradient; given outputs are refused then.
    The weights' gradients are sums in an order that does not change from call to call.  The gradients
    cannot be differentiated again, and forward-mode gradients are refused.  A backward pass may be captured
    into a CUDA graph; no eager graph of the same leaves (an output kept from a warm-up step) may live then, as
    autograd would wait for the stream that it ran on."""
    import torch
    index = _index(q, "q")
    if axes is not None and type(axes) is not tuple:
        axes = tuple(axes)
    _no_tangents("norm_rotary", q, k, q_weight, k_weight)
    if (q.requires_grad or (k is not None and k.requires_grad)
            or (q_weight is not None and q_weight.requires_grad)
            or (k_weight is not None and k_weight.requires_grad)) and torch.is_grad_enabled():
        if q_out is not None or k_out is not None:
            raise ValueError("q_out and k_out cannot be given where a gradient is required")
        if not all(t is None or (t.dim() == 3 and t.shape[1] and t.shape[2]) for t in (q, k)):
            raise ValueError("a gradient needs heads of q and, where it is given, of k")
        if index != torch.cuda.current_device():
            return _elsewhere(index, norm_rotary, q, k, q_weight, k_weight, positions, table, eps=eps,
                              axes=axes, interleaved=interleaved, rot_offset=rot_offset, stream=stream)
        return _recorded()(q, k, q_weight, k_weight, positions, table, eps, axes, interleaved,
                           rot_offset, stream)
    if index != torch.cuda.current_device():
        return _elsewhere(index, norm_rotary, q, k, q_weight, k_weight, positions, table, eps=eps,
                          axes=axes, interleaved=interleaved, rot_offset=rot_offset, q_out=q_out,
                          k_out=k_out, stream=stream)
    args = _norm_args(q, k, q_weight, k_weight, positions, table, eps, axes, interleaved, rot_offset, index)
    return _forward(index, args, q, k, q_out, k_out, stream)

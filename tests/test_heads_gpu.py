"""Rotation by several axes, and queries and keys normalised and rotated at once, with their gradients,
against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import heads_plain as plain
import paged_fp8_mqa_gb300 as idx

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
FLOOR = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
U = 2.0 ** -24  # half a unit of float32


def dev():
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().cpu().double().numpy()


def clean(bits=0):
    torch.cuda.synchronize()
    assert idx.device_status(clear=True) == bits


def sections(rot, axes):
    half = rot // 2
    first = half // axes
    return [half - (axes - 1) * first, *[first] * (axes - 1)]


def close(got, ref, name, slack, size=None):
    """Rounded once to the type, after float32 errors of `slack` units of `size`."""
    size = np.abs(ref) if size is None else size
    lim = slack * U * size
    lim = lim + HALF_ULP[name] * (np.abs(ref) + lim) + FLOOR[name]
    err = np.abs(f64(got) - ref)
    assert (err <= lim).all(), float(np.max(err - lim))


# ---- several axes --------------------------------------------------------------------------------

@pytest.mark.parametrize("T,H,D,rot,offset,interleaved,axes,name", [
    (1, 1, 128, 128, 0, False, 3, "bf16"),
    (37, 5, 128, 128, 0, False, 3, "bf16"),
    (33, 3, 128, 64, 64, True, 2, "f16"),
    (9, 17, 64, 32, 0, False, 4, "bf16"),
    (5, 3, 192, 96, 96, False, 3, "f32"),
    (3, 2, 256, 128, 0, True, 3, "bf16"),
    (4, 3, 96, 24, 72, False, 3, "bf16"),   # pairs that do not fill pieces of eight
    (3, 9, 80, 20, 30, False, 3, "f16"),
    (2, 2, 7, 2, 5, True, 1, "f32"),        # odd rows
    (2, 1, 1024, 1024, 0, False, 4, "bf16"),
    (300, 64, 128, 128, 0, False, 3, "bf16"),  # several heads a lane
])
@pytest.mark.parametrize("layout", ["plain", "strided", "in place"])
def test_rotary_by_axes(T, H, D, rot, offset, interleaved, axes, name, layout):
    clean()
    table = idx.rotary_table(600, rot)
    g = gen(T * 1000 + D)
    base = torch.randn(T, H + 1, D + 8, generator=g).to(DTYPES[name]).to(dev())
    x = base[:, 1:, :D] if layout == "strided" else base[:, :H, :D].contiguous()
    pos = torch.randint(600, (axes, T + 3), generator=g, dtype=torch.int32)[:, :T]
    pos[:, 0] = 599
    pair_axis = idx.rotary_axes(sections(rot, axes), in_turn=H % 2 == 1)
    keep = x.clone()
    y = idx.rotary(x, pos.to(dev()), table, axes=pair_axis, interleaved=interleaved, rot_offset=offset,
                   out=x if layout == "in place" else None)
    clean()
    assert (y.data_ptr() == x.data_ptr()) == (layout == "in place")
    if layout != "in place":
        assert torch.equal(x, keep)
    ref = plain.rotate_axes(f64(keep), pos.tolist(), pair_axis, f64(table), interleaved, offset)
    # Two products and a sum in float32, of terms no larger than the pair's largest.
    size = np.abs(f64(keep)).max(-1, keepdims=True) + 0 * ref
    close(y, ref, name, 6, size)


def test_one_axis_and_equal_axes_are_the_rotation():
    table = idx.rotary_table(100, 64)
    g = gen(5)
    x = torch.randn(20, 6, 64, generator=g).bfloat16().to(dev())
    pos = torch.randint(100, (20,), generator=g, dtype=torch.int32).to(dev())
    want = idx.rotary(x, pos, table)
    axes = idx.rotary_axes((10, 11, 11))
    assert torch.equal(idx.rotary(x, pos.expand(3, 20), table, axes=axes), want)
    assert torch.equal(idx.rotary(x, pos[None], table, axes=[0] * 32), want)


def test_rotary_by_axes_is_undone_and_recorded():
    table = idx.rotary_table(100, 32)
    g = gen(7)
    x = torch.randn(9, 4, 48, generator=g).to(dev()).requires_grad_()
    w = torch.randn(9, 4, 48, generator=g).to(dev())
    pos = torch.randint(100, (3, 9), generator=g, dtype=torch.int32).to(dev())
    axes = idx.rotary_axes((4, 6, 6), in_turn=True)
    y = idx.rotary(x, pos, table, axes=axes, rot_offset=16)
    back = idx.rotary(y.detach(), pos, table, axes=axes, rot_offset=16, inverse=True)
    assert (back - x.detach()).abs().max() <= 16 * U * x.detach().abs().max()
    grad, = torch.autograd.grad(y, x, w)
    ref = plain.rotate_axes(f64(w), pos.tolist(), axes, f64(table), False, 16, back=True)
    close(grad, ref, "f32", 6, np.abs(f64(w)).max() + 0 * ref)


@pytest.mark.parametrize("D,rot,offset,interleaved", [(64, 32, 0, False), (64, 64, 0, True), (48, 20, 8, False)])
def test_pairs_past_the_table_stay_to_the_bit(D, rot, offset, interleaved):
    clean()
    table = idx.rotary_table(10, rot)
    x = torch.randn(4, 3, D, generator=gen(1)).to(dev())
    x[1, 0, offset] = math.inf
    pos = torch.tensor([[3, 10, 2, 9], [1, -1, 5, 2 ** 30]], dtype=torch.int32)
    axes = idx.rotary_axes(sections(rot, 2))
    y = idx.rotary(x, pos.to(dev()), table, axes=axes, interleaved=interleaved, rot_offset=offset)
    clean(idx.IDX_DEV_BAD_POSITION)
    assert torch.equal(y[1], x[1])
    ref = plain.rotate_axes(f64(x)[[0, 2, 3]], pos[:, [0, 2, 3]].tolist(), axes, f64(table), interleaved, offset)
    close(y[[0, 2, 3]], ref, "f32", 6, 6.0 + 0 * ref)
    second = np.array([a == 1 for a in axes])
    half = rot // 2
    i = np.flatnonzero(second)
    at = offset + (2 * i if interleaved else i)
    assert torch.equal(y[3][:, at], x[3][:, at])
    assert torch.equal(y[3][:, at + (1 if interleaved else half)], x[3][:, at + (1 if interleaved else half)])


# ---- norms ---------------------------------------------------------------------------------------

def heads_case(T, H, Hkv, D, rot, offset, interleaved, axes, name, wname, layout="views", seed=0):
    g = gen(seed + T * 100 + D)
    dt = DTYPES[name]
    qkv = torch.randn(T, H + 2 * Hkv, D + (8 if layout == "gaps" else 0), generator=g).to(dt).to(dev())
    q, k = qkv[:, :H, :D], qkv[:, H:H + Hkv, :D]
    if layout == "plain":
        q, k = q.contiguous(), k.contiguous()
    if layout == "odd":  # no 16-byte rows
        q, k = (torch.randn(T, n, D + 1, generator=g).to(dt).to(dev())[:, :, 1:] for n in (H, Hkv))
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(DTYPES[wname]).to(dev()) for _ in range(2)]
    table = idx.rotary_table(500, rot) if rot else None
    pos = torch.randint(500, (axes, T), generator=g, dtype=torch.int32) if rot else None
    pair_axis = idx.rotary_axes(sections(rot, axes)) if axes > 1 else None
    how = dict(axes=pair_axis, interleaved=interleaved, rot_offset=offset)
    at = None if pos is None else (pos if axes > 1 else pos[0]).to(dev())
    plain_how = (None if pos is None else pos.tolist(), pair_axis or (0,) * (rot // 2),
                 None if table is None else f64(table), interleaved, offset)
    return q, k, w, at, table, how, plain_how


def turned(x, plain_how, back=False):
    return x if plain_how[2] is None else plain.rotate_axes(x, *plain_how, back=back)


def check_norm(x, w, y, plain_how, name, eps=1e-6):
    n = plain.norm(f64(x), f64(w), eps)
    ref = turned(n, plain_how)
    # The mean of squares is a float32 sum of D terms in a tree of at most 16 + 5 steps (32 a lane for
    # the widest), half of whose error the root keeps; the root, its product, the weight's: 4 more; the
    # rotation 6 of the pair's largest.
    close(y, ref, name, 64, np.abs(n).max(-1, keepdims=True) + 0 * ref)


HEADS = [  # T, H, Hkv, D, rot, offset, interleaved, axes, dtype, weights
    (1, 1, 1, 128, 128, 0, False, 1, "bf16", "bf16"),
    (37, 6, 2, 128, 128, 0, False, 1, "bf16", "f32"),
    (33, 3, 1, 128, 64, 64, True, 3, "f16", "f16"),
    (9, 17, 3, 64, 32, 32, False, 1, "bf16", "bf16"),
    (5, 3, 2, 192, 48, 144, False, 3, "f32", "f32"),
    (3, 2, 1, 256, 256, 0, True, 1, "bf16", "f32"),
    (4, 3, 2, 96, 24, 0, False, 3, "bf16", "bf16"),  # pairs that do not fill pieces of eight
    (3, 5, 1, 80, 20, 30, True, 1, "f16", "f32"),
    (2, 3, 2, 7, 4, 1, False, 1, "f32", "f32"),
    (2, 1, 1, 1000, 500, 0, False, 2, "bf16", "bf16"),
    (11, 4, 2, 128, 0, 0, False, 1, "bf16", "bf16"),  # no rotation
    (700, 33, 5, 128, 128, 0, False, 1, "bf16", "bf16"),  # several heads a lane, odd numbers of them
]


@pytest.mark.parametrize("T,H,Hkv,D,rot,offset,interleaved,axes,name,wname", HEADS)
@pytest.mark.parametrize("layout", ["views", "plain", "gaps", "odd"])
def test_norm_rotary(T, H, Hkv, D, rot, offset, interleaved, axes, name, wname, layout):
    clean()
    q, k, w, pos, table, how, ph = heads_case(T, H, Hkv, D, rot, offset, interleaved, axes, name, wname, layout)
    keep = q.clone(), k.clone()
    qo, ko = idx.norm_rotary(q, k, *w, pos, table, **how)
    clean()
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])
    check_norm(q, w[0], qo, ph, name)
    check_norm(k, w[1], ko, ph, name)
    # One of the two alone; in place.
    alone, none = idx.norm_rotary(q, None, w[0], None, pos, table, **how)
    assert none is None and torch.equal(alone, qo)
    same = idx.norm_rotary(q, k, *w, pos, table, q_out=q, k_out=k, **how)
    assert same[0] is q and torch.equal(q, qo) and torch.equal(k, ko)


def test_norm_without_weights_and_of_special_rows():
    """No weights; a row of zeros (eps alone), tiny and large rows, a NaN that stays in its head."""
    clean()
    q = torch.randn(6, 4, 64, generator=gen(3)).to(dev())
    q[0, 1] = 0
    q[1] *= 1e-12
    q[2] *= 1e12
    q[3, 2, 5] = math.nan
    y, _ = idx.norm_rotary(q, None, eps=1e-5)
    clean()
    ok = torch.ones(6, 4, dtype=torch.bool)
    ok[3, 2] = False
    assert torch.isnan(y[3, 2]).all() and (y[0, 1] == 0).all()
    ref = plain.norm(f64(q)[ok.numpy()][:, None], 1.0, 1e-5)[:, 0]
    close(y[ok.to(dev())], ref, "f32", 64, np.abs(ref).max(-1, keepdims=True) + 0 * ref)


def check_gradients(x, w, g, dx, dw, ph, name, wname, eps=1e-6):
    gr = turned(f64(g), ph, back=True)
    X, W = f64(x), f64(w)
    rdx, rdw = plain.norm_gradients(X, W, eps, gr)
    r = 1 / np.sqrt((X * X).mean(-1, keepdims=True) + eps)
    # Every term of dx is at most r |g w| or r^3 |x| mean|g w x|, each with the forward's errors.
    size = r * np.abs(gr * W).max(-1, keepdims=True) + np.abs(X) * r ** 3 * np.abs(gr * W * X).mean(-1, keepdims=True)
    close(dx, rdx, name, 96, size + 0 * rdx)
    # A float32 sum in registers of at most rows / lanes terms, then of the blocks in 64 bits.
    terms = np.abs(gr * X * r).sum((0, 1))
    close(dw, rdw, wname, 64 + X.shape[0] * X.shape[1] / 16, terms)


@pytest.mark.parametrize("T,H,Hkv,D,rot,offset,interleaved,axes,name,wname", HEADS)
@pytest.mark.parametrize("layout", ["views", "odd"])
def test_norm_rotary_gradients(T, H, Hkv, D, rot, offset, interleaved, axes, name, wname, layout):
    clean()
    q, k, w, pos, table, how, ph = heads_case(T, H, Hkv, D, rot, offset, interleaved, axes, name, wname, layout)
    g = gen(11)
    gq, gk = (torch.randn(t.shape, generator=g).to(t.dtype).to(dev()) for t in (q, k))
    leaves = [t.detach().requires_grad_() for t in (q, k, *w)]
    out = idx.norm_rotary(*leaves, pos, table, **how)
    dq, dk, dqw, dkw = torch.autograd.grad(out, leaves, (gq, gk))
    clean()
    check_gradients(q, w[0], gq, dq, dqw, ph, name, wname)
    check_gradients(k, w[1], gk, dk, dkw, ph, name, wname)
    # The same bits each time.
    out = idx.norm_rotary(*leaves, pos, table, **how)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dqw, dkw), torch.autograd.grad(out, leaves, (gq, gk))))


def test_norm_rotary_gradients_by_differences():
    """In float32, the derivative along random directions against central differences of the float64
    formula's values (whose step error is h^2) and of the call's own."""
    T, H, D = 3, 2, 32
    q, k, w, pos, table, how, ph = heads_case(T, H, 1, D, 16, 8, True, 3, "f32", "f32", "plain")
    g = gen(13)
    gq = torch.randn(T, H, D, generator=g).to(dev())
    lq, lw = q.detach().requires_grad_(), w[0].detach().requires_grad_()
    y, _ = idx.norm_rotary(lq, None, lw, None, pos, table, **how)
    dq, dw = torch.autograd.grad(y, (lq, lw), gq)
    call = lambda x, ww: (f64(idx.norm_rotary(x, None, ww, None, pos, table, **how)[0]) * f64(gq)).sum()  # noqa: E731
    h = 2.0 ** -6
    for seed in range(4):
        d = torch.randn(T, H, D, generator=gen(seed)).to(dev())
        want = (call(q + h * d, w[0]) - call(q - h * d, w[0])) / (2 * h)
        got = (f64(dq) * f64(d)).sum()
        # Third derivatives of x / rms: below 50 for rows of this size, times h^2 / 6; rounding U / h each.
        assert abs(got - want) <= T * H * D * (50 * h * h / 6 + 4 * U / h)
        e = torch.randn(D, generator=gen(seed)).to(dev())
        want = (call(q, w[0] + e) - call(q, w[0] - e)) / 2  # linear in the weight
        assert abs((f64(dw) * f64(e)).sum() - want) <= T * H * D * 16 * U * 4


def test_gradients_of_what_is_asked_for():
    """A weight alone, one output alone, an expanded gradient (of a sum), no weights, no tokens."""
    q, k, w, pos, table, how, ph = heads_case(7, 4, 2, 64, 32, 0, False, 1, "f32", "f32")
    lw = w[1].detach().requires_grad_()
    out = idx.norm_rotary(q, k, w[0], lw, pos, table, **how)
    assert out[0].grad_fn is not None and out[1].requires_grad
    ones = torch.ones_like(k)
    dw, = torch.autograd.grad(out[1].sum(), lw)
    check_gradients(k, w[1], ones, idx.heads._backward(q, k, *w, pos, table, 1e-6, None, False, 0, torch.zeros_like(q), ones)[1], dw, ph, "f32", "f32")
    lq = q.detach().requires_grad_()
    y, none = idx.norm_rotary(lq, None, None, None, pos, table, **how)
    dq, = torch.autograd.grad(y, lq, ones[:, :1].expand(7, 4, 64))
    check_gradients(q, torch.ones(64), ones[:, :1].expand(7, 4, 64), dq, torch.tensor(plain.norm_gradients(f64(q), 1.0, 1e-6, turned(np.ones((7, 4, 64)), ph, back=True))[1]), ph, "f32", "f32")
    assert none is None
    empty = torch.zeros(0, 4, 64, device=dev(), requires_grad=True)
    lw = w[0].detach().requires_grad_()
    y, _ = idx.norm_rotary(empty, None, lw, None, pos[:0], table, **how)
    dx, dw = torch.autograd.grad(y.sum(), (empty, lw))
    assert dx.shape == (0, 4, 64) and (dw == 0).all()
    with pytest.raises(RuntimeError):  # gradients cannot be differentiated again
        y, _ = idx.norm_rotary(lq, None, None, None, pos, table, **how)
        dq, = torch.autograd.grad(y.sum(), lq, create_graph=True)
        dq.sum().backward()


def test_positions_past_the_table():
    """They leave their rows normalised and not turned, and so do their gradients."""
    clean()
    q, k, w, pos, table, how, ph = heads_case(4, 3, 2, 64, 32, 0, False, 1, "f32", "f32")
    pos[2] = 500
    out = idx.norm_rotary(q, k, *w, pos, table, **how)
    clean(idx.IDX_DEV_BAD_POSITION)
    ph = ([pos.tolist()], *ph[1:])
    check_norm(q, w[0], out[0], ph, "f32")
    check_norm(k, w[1], out[1], ph, "f32")
    g = [torch.randn_like(t) for t in (q, k)]
    dq, dk, dqw, dkw = idx.heads._backward(q, k, *w, pos, table, 1e-6, None, False, 0, *g)
    check_gradients(q, w[0], g[0], dq, dqw, ph, "f32", "f32")
    idx.device_status(clear=True)


def test_on_another_stream_and_in_a_graph():
    q, k, w, pos, table, how, ph = heads_case(40, 8, 2, 128, 128, 0, False, 1, "bf16", "bf16")
    want = idx.norm_rotary(q, k, *w, pos, table, **how)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = idx.norm_rotary(q, k, *w, pos, table, stream=s, **how)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, *w)]
    g = [torch.randn_like(t) for t in want]
    eager = torch.autograd.grad(idx.norm_rotary(*leaves, pos, table, **how), leaves, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = idx.norm_rotary(*leaves, pos, table, **how)
        grads = torch.autograd.grad(out, leaves, g)
    with torch.no_grad():
        leaves[0].mul_(2.0)  # (the norm takes it out again, but for eps and the roundings)
        leaves[0].mul_(0.5)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, eager)) and torch.equal(out[0], want[0])


def test_refusals_of_tensors():
    q, k, w, pos, table, how, _ = heads_case(6, 4, 2, 64, 32, 0, False, 1, "f32", "f32", "plain")
    two = pos.expand(2, 6)
    axes = idx.rotary_axes((8, 8))
    for bad, error in (
            (lambda: idx.norm_rotary(q, k.half(), *w, pos, table), TypeError),
            (lambda: idx.norm_rotary(q, k[:5], *w, pos, table), TypeError),
            (lambda: idx.norm_rotary(q, k, w[0][:32], w[1], pos, table), ValueError),
            (lambda: idx.norm_rotary(q, k, w[0].half(), w[1], pos, table), TypeError),
            (lambda: idx.norm_rotary(q, k, w[0].bfloat16(), w[1].half(), pos, table), TypeError),
            (lambda: idx.norm_rotary(q, None, w[0], w[1], pos, table), ValueError),
            (lambda: idx.norm_rotary(q, k, *w, pos), ValueError),
            (lambda: idx.norm_rotary(q, k, *w, pos[:5], table), ValueError),
            (lambda: idx.norm_rotary(q, k, *w, two, table), ValueError),
            (lambda: idx.norm_rotary(q, k, *w, pos, table, axes=axes), ValueError),
            (lambda: idx.norm_rotary(q, k, *w, two, table, axes=axes[:-1]), ValueError),
            (lambda: idx.norm_rotary(q, k, *w, two.t().contiguous().t(), table, axes=axes), ValueError),
            (lambda: idx.norm_rotary(q, k, *w, pos, table, q_out=k), ValueError),
            (lambda: idx.norm_rotary(q, k, *w, pos, table, q_out=q[:1].expand(6, 4, 64)), ValueError),
            (lambda: idx.norm_rotary(q, k, *w, pos, table, rot_offset=40), idx.IdxError),
            (lambda: idx.norm_rotary(q, k, *w, pos, table, eps=-1.0), idx.IdxError),
            (lambda: idx.norm_rotary(q.requires_grad_(), k, *w, pos, table, q_out=torch.empty_like(q)), ValueError),
            (lambda: idx.norm_rotary(torch.zeros(2, 1, 1040, device=dev())), None),
            (lambda: idx.norm_rotary(torch.zeros(2, 1, 1040, device=dev()), None), idx.IdxError),
            (lambda: idx.rotary(k, two.expand(5, 2, 6)[0], table, axes=axes), None),
            (lambda: idx.rotary(k, pos.expand(5, 6), table, axes=axes), ValueError)):
        if error is None:
            continue
        with pytest.raises(error):
            bad()
    torch.cuda.synchronize()


def test_c_entry_of_the_gradients_without_tokens():
    """No tokens: the weights' gradients are zeros."""
    w = torch.ones(64, device=dev())
    g = [torch.full((64,), 5.0, device=dev()) for _ in range(2)]
    need = idx.idx_norm_rotary_workspace_bytes(64)
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    p = w.data_ptr()
    rows = (p, 128, 64)
    assert idx.idx_norm_rotary_backward(*rows, 2, *rows, 1, idx.IDX_DTYPE_F32, 0, 64, p, p, idx.IDX_DTYPE_F32,
                                        1e-6, None, 0, None, 1, None, 0, 0, 0, 0, *rows, *rows, p, p,
                                        g[0].data_ptr(), g[1].data_ptr(), ws.data_ptr(), need, None) == 0
    clean()
    assert (g[0] == 0).all() and (g[1] == 0).all()


def test_c_entry_of_the_gradients_without_heads():
    """No heads: the same."""
    w = torch.ones(64, device=dev())
    g = torch.full((64,), 5.0, device=dev())
    need = idx.idx_norm_rotary_workspace_bytes(64)
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    p = w.data_ptr()
    rows, none = (p, 64, 64), (None, 0, 0)
    assert idx.idx_norm_rotary_backward(*rows, 0, *none, 0, idx.IDX_DTYPE_F32, 3, 64, p, None, idx.IDX_DTYPE_F32,
                                        1e-6, None, 0, None, 1, None, 0, 0, 0, 0, *rows, *none, p, None,
                                        g.data_ptr(), None, ws.data_ptr(), need, None) == 0
    clean()
    assert (g == 0).all()


def test_axes_that_can_be_read_only_once():
    q, k, w, pos, table, how, ph = heads_case(5, 4, 2, 64, 32, 0, False, 3, "f32", "f32")
    want = [torch.autograd.grad(y, x, torch.ones_like(y)) for x in (q.detach().requires_grad_(),) for y in
            (idx.norm_rotary(x, None, w[0], None, pos, table, **how)[0], idx.rotary(x, pos, table, **how))]
    x = q.detach().requires_grad_()
    for f, (dx,) in zip((lambda axes: idx.norm_rotary(x, None, w[0], None, pos, table, axes=axes)[0],
                         lambda axes: idx.rotary(x, pos, table, axes=axes)), want):
        y = f(a for a in how["axes"])
        assert torch.equal(torch.autograd.grad(y, x, torch.ones_like(y))[0], dx)


@pytest.mark.parametrize("name,wname", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
def test_c_entry_of_the_gradients_without_keys_heads(name, wname):
    """No heads of k, whose weight and its gradient are given: the sum over nothing is 0, q's is its own."""
    T, H, D = 5, 3, 64
    x, g = (torch.randn(T, H, D, generator=gen(i)).to(DTYPES[name]).to(dev()) for i in (1, 2))
    w = torch.ones(D, dtype=DTYPES[wname], device=dev())
    dqw, dkw = (torch.full((D,), 5.0, dtype=w.dtype, device=dev()) for _ in range(2))
    dx = torch.empty_like(x)
    need = idx.idx_norm_rotary_workspace_bytes(D)
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    rows = lambda t: (t.data_ptr(), H * D, D)  # noqa: E731
    none, code = (None, 0, 0), {"f32": idx.IDX_DTYPE_F32, "f16": idx.IDX_DTYPE_F16, "bf16": idx.IDX_DTYPE_BF16}
    for want_q in (True, False):
        assert idx.idx_norm_rotary_backward(
            *rows(x), H, *none, 0, code[name], T, D, w.data_ptr(), w.data_ptr(), code[wname], 1e-6, None, 0,
            None, 1, None, 0, 0, 0, 0, *rows(g), *none, dx.data_ptr(), None,
            dqw.data_ptr() if want_q else None, dkw.data_ptr(), ws.data_ptr(), need, None) == 0
        clean()
        assert (dkw == 0).all()
        check_gradients(x, w, g, dx, dqw, (None, None, None, False, 0), name, wname)
        dkw.fill_(5.0)


@pytest.mark.parametrize("kind", ["the same", "copies", "on the host", "positions moved", "q moved", "weight moved"])
def test_gradients_with_hooks_on_what_is_saved(kind):
    """Tensors that hooks put in the place of the saved ones are read as they lie: at other addresses, or at the
    same ones with other strides."""
    clean()
    T, H, Hkv, D = 9, 4, 2, 64
    q, k, w, _, table, how, ph = heads_case(T, H, Hkv, D, 32, 0, False, 2, "f32", "f32")
    g = gen(3)
    room = torch.randint(500, (2 * (T + 7),), generator=g, dtype=torch.int32).to(dev())
    pos = room.view(2, T + 7)[:, :T]
    wide = torch.empty(T * H * 2 * D, device=dev())
    wide_q = wide.view(T, H, 2 * D)[:, :, :D].copy_(q)
    wide_w = torch.empty(2 * D, device=dev())
    wide_w[:D] = w[0]
    grads = [torch.randn(t.shape, generator=g).to(dev()) for t in (q, k)]
    leaves = [t.detach().requires_grad_() for t in (wide_q, k, wide_w[:D], w[1])]
    call = lambda: idx.norm_rotary(*leaves, pos, table, **how)  # noqa: E731
    want = torch.autograd.grad(call(), leaves, grads)
    ph = (pos.tolist(), *ph[1:])
    check_gradients(q, w[0], grads[0], want[0], want[2], ph, "f32", "f32")

    def pack(t):
        moved = {"positions moved": pos, "q moved": wide_q, "weight moved": wide_w}.get(kind)
        if kind == "copies" or (moved is not None and t.data_ptr() == moved.data_ptr()):
            return t.clone()
        return t.cpu() if kind == "on the host" else t

    def unpack(t):
        if kind == "on the host":
            return t.to(dev())
        if kind == "positions moved" and t.dtype == torch.int32:
            return room[:2 * T].copy_(t.reshape(-1)).view(2, T)
        if kind == "q moved" and t.dim() == 3 and t.shape[1:] == (H, D) and t.data_ptr() != wide.data_ptr():
            return wide[:T * H * D].copy_(t.reshape(-1)).view(T, H, D)
        if kind == "weight moved" and t.dim() == 1 and t.data_ptr() != w[1].data_ptr():
            wide_w[::2] = t
            return wide_w[::2]
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, unpack):
        out = call()
    if kind == "weight moved":
        with pytest.raises(ValueError, match="contiguous"):  # (as a call with such a weight)
            torch.autograd.grad(out, leaves, grads)
        return
    with torch.no_grad():
        got = torch.autograd.grad(out, leaves, grads)
    clean()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_forward_mode_gradients_are_refused():
    """A dual tensor, which does not require a gradient, is refused where its tangent would be lost; what has
    no tangent runs while a dual level is open."""
    from torch.autograd import forward_ad
    q, k, w, pos, table, how, _ = heads_case(5, 4, 2, 64, 32, 0, False, 3, "f32", "f32", "plain")
    want = idx.norm_rotary(q, k, *w, pos, table, **how)
    turned_q = idx.rotary(q, pos, table, **how)
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for at in range(4):
            args = [q, k, *w]
            args[at] = dual(args[at])
            with torch.no_grad(), pytest.raises(NotImplementedError, match="norm_rotary"):
                idx.norm_rotary(*args, pos, table, **how)
        for more in (dict(how), dict(how, out=torch.empty_like(q))):
            with pytest.raises(NotImplementedError, match="rotary"):
                idx.rotary(dual(q), pos, table, **more)
        with pytest.raises(NotImplementedError, match="rotary"):
            idx.rotary(dual(q), pos[0].contiguous(), table)
        assert all(torch.equal(a, b) for a, b in zip(idx.norm_rotary(q, k, *w, pos, table, **how), want))
        assert torch.equal(idx.rotary(q, pos, table, **how), turned_q)
        assert idx.norm_rotary(q, None, None, None)[1] is None
    torch.cuda.synchronize()


@pytest.mark.parametrize("D,rot,offset,interleaved,name", [
    (64, 0, 0, False, "f32"), (128, 64, 32, False, "bf16"), (128, 64, 32, True, "f16"),
    (192, 96, 0, False, "bf16"), (96, 24, 0, True, "f32"), (80, 20, 30, False, "bf16")])
def test_what_is_not_finite_in_a_weight_stays_with_its_element(D, rot, offset, interleaved, name):
    """An infinite and a NaN weight of elements that are not turned, in the rotated part of a token past the
    table too: those elements show it, all others are what they are without."""
    clean()
    q, k, w, pos, table, how, _ = heads_case(7, 3, 2, D, rot, offset, interleaved, 1, name, "f32", "plain")
    odd = [d for d in range(D) if not offset <= d < offset + rot][1::5]
    plain_w = [x.clone() for x in w]
    for x in w:
        x[odd[0]], x[odd[1]], x[odd[2]] = math.inf, math.nan, -math.inf
    ok = torch.ones(D, dtype=torch.bool)
    ok[odd[:3]] = False
    ok = ok.to(dev())
    got = idx.norm_rotary(q, k, *w, pos, table, **how)
    want = idx.norm_rotary(q, k, *plain_w, pos, table, **how)
    clean()
    for g, e in zip(got, want):
        assert torch.equal(g[:, :, ok], e[:, :, ok]) and not torch.isfinite(g[:, :, ~ok]).any()
    if rot:
        pos[:] = 500  # (past the table: nothing is turned)
        w[0][offset + 1] = math.inf
        ok[offset + 1] = False
        got = idx.norm_rotary(q, None, w[0], None, pos, table, **how)[0]
        want = idx.norm_rotary(q, None, plain_w[0], None, pos, table, **how)[0]
        clean(idx.IDX_DEV_BAD_POSITION)
        assert torch.equal(got[:, :, ok], want[:, :, ok]) and not torch.isfinite(got[:, :, ~ok]).any()

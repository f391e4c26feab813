"""Rotation by several axes and normalised heads at the sizes where a group of lanes walks several heads (2, 4,
8 or 16 of them, with loads ahead), where every smaller call takes one; and past 2^31 elements.  Against the
formulas in 64 bits, in elementary torch operations."""
import pytest
import torch

import paged_fp8_mqa_gb300 as idx

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
FLOOR = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
U = 2.0 ** -24  # half a unit of float32
EPS = 1e-6


def dev():
    return torch.device("cuda:0")


def clean(bits=0):
    torch.cuda.synchronize()
    assert idx.device_status(clear=True) == bits


def walk_of(T, heads, D):
    """Heads that a group of lanes takes: 16, halved while that leaves fewer than 8192 warps."""
    lanes = 4 if D <= 64 else 8 if D <= 128 else 16
    walk = 16
    while walk > 1 and T * (heads // walk) * lanes // 32 < 8192:
        walk //= 2
    return walk


def close(got, ref, name, slack, size):
    """Rounded once to the type, after float32 errors of `slack` units of `size`."""
    lim = slack * U * size
    lim = lim + HALF_ULP[name] * (ref.abs() + lim) + FLOOR[name]
    err = (got.double() - ref).abs()
    assert (err <= lim).all(), float((err - lim).max())


def rotate(x, pos, axes, table, interleaved, offset, back=False):
    """x [T, H, D] float64, positions [A, T]: pair i turned by its own axis' position."""
    half = table.shape[1]
    of = torch.tensor(axes, device=x.device)
    cs = table.double()[pos[of].long(), torch.arange(half, device=x.device)[:, None]]  # [half, T, 2]
    c, s = (t.t()[:, None] for t in (cs[..., 0], cs[..., 1] * (-1 if back else 1)))
    i = torch.arange(half, device=x.device)
    a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + half + i)
    y = x.clone()
    y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
    y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def inputs(T, H, Hkv, D, rot, axes, name, wname, layout, seed):
    g = torch.Generator(dev()).manual_seed(seed)
    gap = 8 if layout == "gaps" else 0
    qkv = torch.randn(T, H + 2 * Hkv, D + gap, generator=g, device=dev()).to(DTYPES[name])
    q, k = qkv[:, :H, :D], qkv[:, H:H + Hkv, :D]
    w = [(1 + 0.3 * torch.randn(D, generator=g, device=dev())).to(DTYPES[wname]) for _ in range(2)]
    pos = torch.randint(500, (axes, T + 5), generator=g, device=dev(), dtype=torch.int32)[:, :T]
    sections = [rot // 2 - (axes - 1) * (rot // 2 // axes), *[rot // 2 // axes] * (axes - 1)]
    return q, k, w, pos, idx.rotary_table(500, rot), idx.rotary_axes(sections), g


CASES = [  # the walk, T, H, Hkv, D, rot, offset, interleaved, axes, dtype, weights, layout
    (2, 1201, 64, 8, 128, 128, 0, False, 1, "bf16", "bf16", "views"),
    (4, 4099, 33, 5, 128, 128, 0, False, 3, "bf16", "bf16", "views"),
    (8, 4099, 64, 9, 128, 64, 64, True, 2, "f16", "f32", "gaps"),
    (16, 8201, 70, 5, 128, 128, 0, False, 1, "bf16", "f32", "views"),
    (4, 5101, 50, 3, 64, 32, 32, False, 1, "f16", "f16", "gaps"),
    (16, 16411, 67, 0, 64, 64, 0, True, 3, "bf16", "bf16", "views"),
    (16, 16411, 20, 3, 192, 96, 96, False, 3, "bf16", "bf16", "views"),  # 12 lanes of 16
    (8, 8209, 17, 2, 256, 256, 0, True, 1, "f32", "f32", "gaps"),
    (4, 4099, 33, 5, 128, 64, 0, False, 2, "f32", "f32", "views"),
    (2, 3001, 13, 1, 224, 32, 64, True, 1, "f16", "f32", "gaps"),        # 14 lanes of 16
    (16, 8200, 40, 40, 80, 16, 48, False, 4, "bf16", "f32", "views"),    # 5 lanes of 8
]
IDS = [f"{c[1]}x{c[2]}+{c[3]}x{c[4]}-{c[9]}" for c in CASES]


@pytest.mark.parametrize("walk,T,H,Hkv,D,rot,offset,interleaved,axes,name,wname,layout", CASES, ids=IDS)
def test_norm_rotary_walks(walk, T, H, Hkv, D, rot, offset, interleaved, axes, name, wname, layout):
    assert walk_of(T, H + Hkv, D) == walk
    clean()
    q, k, w, pos, table, pair_axis, _ = inputs(T, H, Hkv, D, rot, axes, name, wname, layout, T + D)
    how = dict(axes=pair_axis if axes > 1 else None, interleaved=interleaved, rot_offset=offset)
    at = pos if axes > 1 else pos[0]
    out = idx.norm_rotary(q, k, *w, at, table, **how)
    clean()
    for x, ww, y in zip((q, k), w, out):
        if x.shape[1]:
            n = x.double() * (x.double().square().mean(-1, keepdim=True) + EPS).rsqrt() * ww.double()
            ref = rotate(n, pos, pair_axis, table, interleaved, offset)
            # As for the small sizes: 16 + 5 steps of the sum, the root, three products, the rotation.
            close(y, ref, name, 64, n.abs().amax(-1, keepdim=True))
            del n, ref
    same = idx.norm_rotary(q, k, *w, at, table, q_out=q, k_out=k, **how)
    clean()
    assert torch.equal(same[0], out[0]) and torch.equal(same[1], out[1])


@pytest.mark.parametrize("walk,T,H,Hkv,D,rot,offset,interleaved,axes,name,wname,layout", CASES, ids=IDS)
def test_rotary_by_axes_walks(walk, T, H, Hkv, D, rot, offset, interleaved, axes, name, wname, layout):
    clean()
    axes = max(axes, 2)
    H += Hkv  # (so that the walk is the same)
    q, _, _, pos, table, pair_axis, _ = inputs(T, H, 0, D, rot, axes, name, wname, layout, T + D + 1)
    assert walk_of(T, H, D) == walk
    how = dict(axes=pair_axis, interleaved=interleaved, rot_offset=offset)
    pos[1, 7] = 500  # (past the table: the pairs of that axis stay)
    y = idx.rotary(q, pos, table, **how)
    clean(idx.IDX_DEV_BAD_POSITION)
    few = idx.rotary(q[5:9], pos[:, 5:9], table, **how)
    idx.device_status(clear=True)
    assert torch.equal(y[5:9], few)
    there = torch.arange(T, device=dev()) != 7
    pos[1, 7] = 0
    ref = rotate(q.double(), pos, pair_axis, table, interleaved, offset)
    close(y[there], ref[there], name, 6, q[there].double().abs().amax(-1, keepdim=True))
    back = idx.rotary(y, pos, table, inverse=True, **how)
    ref = rotate(y.double(), pos, pair_axis, table, interleaved, offset, back=True)
    close(back, ref, name, 6, y.double().abs().amax(-1, keepdim=True))
    idx.rotary(q, pos, table, out=q, **how)
    clean()
    assert torch.equal(q[there], y[there])


@pytest.mark.parametrize("walk,T,H,Hkv,D,rot,offset,interleaved,axes,name,wname,layout", CASES, ids=IDS)
def test_norm_rotary_gradients_walk(walk, T, H, Hkv, D, rot, offset, interleaved, axes, name, wname, layout):
    """(Gradients walk at most four heads, and these sizes all do.)"""
    clean()
    q, k, w, pos, table, pair_axis, g = inputs(T, H, Hkv, D, rot, axes, name, wname, layout, T + D + 2)
    lanes = 4 if D <= 64 else 8 if D <= 128 else 16
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    groups = 4 * sms * (128 // lanes)
    how = dict(axes=pair_axis if axes > 1 else None, interleaved=interleaved, rot_offset=offset)
    at = pos if axes > 1 else pos[0]
    if not Hkv:
        k, w = None, (w[0], None)
    grads = [None if x is None else torch.randn(x.shape, generator=g, device=dev()).to(x.dtype) for x in (q, k)]
    leaves = [None if t is None else t.detach().requires_grad_() for t in (q, k, *w)]
    out = idx.norm_rotary(*leaves, at, table, **how)
    asked = [t for t in leaves if t is not None]
    got = torch.autograd.grad([y for y in out if y is not None], asked, [x for x in grads if x is not None])
    clean()
    n = len(asked) // 2
    for x, ww, dy, dx, dw in zip((q, k), w, grads, got[:n], got[n:]):
        X, W = x.double(), ww.double()
        G = rotate(dy.double(), pos, pair_axis, table, interleaved, offset, back=True)
        r = (X.square().mean(-1, keepdim=True) + EPS).rsqrt()
        gw = G * W
        mean = (gw * X).mean(-1, keepdim=True)
        # Every term of dx is at most r |g w| or r^3 |x| mean|g w x|, each with the forward's errors.
        size = r * gw.abs().amax(-1, keepdim=True) + X.abs() * r ** 3 * (gw * X).abs().mean(-1, keepdim=True)
        close(dx, r * gw - X * r ** 3 * mean, name, 96, size)
        del gw, size
        # A lane's float32 sum over its rows, a block's over its groups (at most 32), the blocks' exactly but
        # for 2^-24 of it; each term with the forward's errors.
        rows = 1.1 * T * (H + Hkv) / groups + 8
        close(dw, (G * X * r).sum((0, 1)), wname, 64 + rows + 32 + 4, (G * X * r).abs().sum((0, 1)))
        del X, G, r, mean


def test_norm_rotary_and_its_gradients_past_32_bits_of_elements():
    """More than 2^31 elements of q: the last tokens against their own call, the weight's gradient against the
    formula's sum."""
    T, H, D = 140_001, 120, 128
    assert T * H * D > 2 ** 31
    g = torch.Generator(dev()).manual_seed(5)
    table = idx.rotary_table(500, 64)
    pos = torch.randint(500, (T,), generator=g, device=dev(), dtype=torch.int32)
    w = (1 + 0.3 * torch.randn(D, generator=g, device=dev())).requires_grad_()
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device=dev())
    dy = torch.empty_like(q)
    for t in (q, dy):
        for i in range(0, T, 20_000):
            t[i:i + 20_000] = torch.randn(t[i:i + 20_000].shape, generator=g, device=dev())
    leaf = q.requires_grad_()
    clean()
    y, _ = idx.norm_rotary(leaf, None, w, None, pos, table)
    dx, dw = torch.autograd.grad(y, (leaf, w), dy)
    clean()
    y = y.detach()
    want = torch.zeros(D, dtype=torch.float64, device=dev())
    terms = torch.zeros_like(want)
    pairs = (0,) * 32
    with torch.no_grad():
        for i in range(0, T, 10_000):
            at = slice(i, i + 10_000)
            X, P = q[at].double(), pos[None, at]
            r = (X.square().mean(-1, keepdim=True) + EPS).rsqrt()
            n = X * r * w.double()
            G = rotate(dy[at].double(), P, pairs, table, False, 0, back=True)
            want += (G * X * r).sum((0, 1))
            terms += (G * X * r).abs().sum((0, 1))
            if i in (0, 130_000, 140_000):
                close(y[at], rotate(n, P, pairs, table, False, 0), "bf16", 64, n.abs().amax(-1, keepdim=True))
                gw = G * w.double()
                size = r * gw.abs().amax(-1, keepdim=True) + X.abs() * r ** 3 * (gw * X).abs().mean(-1, keepdim=True)
                close(dx[at], r * gw - X * r ** 3 * (gw * X).mean(-1, keepdim=True), "bf16", 96, size)
            del X, r, n, G
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    close(dw, want, "f32", 64 + 1.1 * T * H / (4 * sms * 16) + 8 + 16 + 4, terms)


@pytest.mark.parametrize("D,name", [(64, "f32"), (80, "bf16"), (128, "bf16")])
def test_positions_with_a_gap_between_axes(D, name):
    """norm_rotary and its gradients read positions [axes, T] by the stride between axes."""
    T, H, Hkv = 9, 4, 2
    q, k, w, pos, table, axes, g = inputs(T, H, Hkv, D, 32, 3, name, "f32", "views", 7)
    assert pos.stride(0) == T + 5
    dense = pos.contiguous()
    grads = [torch.randn(x.shape, generator=g, device=dev()).to(x.dtype) for x in (q, k)]
    leaves = [t.detach().requires_grad_() for t in (q, k, *w)]
    results = []
    for p in (pos, dense):
        out = idx.norm_rotary(*leaves, p, table, axes=axes)
        results.append([*out, *torch.autograd.grad(out, leaves, grads)])
    clean()
    assert all(torch.equal(a, b) for a, b in zip(*results))
    one = idx.norm_rotary(*(t.detach() for t in leaves), pos[:1].expand(3, T), table, axes=axes)
    single = idx.norm_rotary(*(t.detach() for t in leaves), pos[0], table)
    assert torch.equal(one[0], single[0]) and torch.equal(one[1], single[1])


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,Hkv,D,layout", [(1201, 64, 8, 128, "views"), (9, 5, 2, 64, "views"),
                                              (9, 5, 2, 192, "odd"), (4, 3, 1, 72, "views")])
def test_rows_whose_squares_leave_float32(T, H, Hkv, D, layout, name):
    """Rows of 2^100, 2^124 and 2^-100 among ordinary ones, whose squares are infinite or 0 in float32: the
    norm and its gradients are the formula's; a row of zeros gives zeros (with eps) or NaN (0 / 0)."""
    clean()
    g = torch.Generator(dev()).manual_seed(T + D)
    table, axes = idx.rotary_table(500, 32), (0,) * 16
    pos = torch.randint(500, (1, T), generator=g, device=dev(), dtype=torch.int32)
    extra = 1 if layout == "odd" else 0  # (rows that are not 16-byte aligned take the general kernels)

    def rows(n, powers):
        x = torch.randn(T, n, D + extra, generator=g, device=dev())
        at = torch.randint(len(powers), (T, n, 1), generator=g, device=dev())
        return (x * torch.tensor([2.0 ** p for p in powers], device=dev())[at]).to(DTYPES[name])[:, :, extra:]

    w = [1 + 0.3 * torch.randn(D, generator=g, device=dev()) for _ in range(2)]
    for powers, eps in (((0, 100, 124, 0), 1e-6), ((0, 100, 124, -100, -100), 0.0)):
        q, k = rows(H, powers), rows(Hkv, powers)
        out = idx.norm_rotary(q, k, *w, pos[0], table, eps=eps)
        clean()
        for x, ww, y in zip((q, k), w, out):
            n = x.double() * (x.double().square().mean(-1, keepdim=True) + eps).rsqrt() * ww.double()
            close(y, rotate(n, pos, axes, table, False, 0), name, 64, n.abs().amax(-1, keepdim=True))
    for powers, eps in (((0, 80, 100, 0), 1e-6), ((0, 100, -100, -80), 0.0)):
        q, k = rows(H, powers), rows(Hkv, powers)
        grads = [torch.randn(x.shape, generator=g, device=dev()).to(x.dtype) for x in (q, k)]
        leaves = [t.detach().requires_grad_() for t in (q, k, *w)]
        got = torch.autograd.grad(idx.norm_rotary(*leaves, pos[0], table, eps=eps), leaves, grads)
        clean()
        for x, ww, dy, dx, dw in zip((q, k), w, grads, got[:2], got[2:]):
            X, W = x.double(), ww.double()
            G = rotate(dy.double(), pos, axes, table, False, 0, back=True)
            r = (X.square().mean(-1, keepdim=True) + eps).rsqrt()
            gw = G * W
            size = r * gw.abs().amax(-1, keepdim=True) + X.abs() * r ** 3 * (gw * X).abs().mean(-1, keepdim=True)
            close(dx, r * gw - X * r ** 3 * (gw * X).mean(-1, keepdim=True), name, 96, size)
            close(dw, (G * X * r).sum((0, 1)), "f32", 64 + 32 + T, (G * X * r).abs().sum((0, 1)))
    q = rows(H, (0, 124))
    q[0, 0] = 0
    q[1, 0, 3], q[1, 1, 3] = float("inf"), float("nan")
    y, _ = idx.norm_rotary(q, None, eps=1e-6)
    assert (y[0, 0] == 0).all() and torch.isnan(y[1, 1]).all()
    assert torch.isnan(y[1, 0, 3]) and (torch.cat((y[1, 0, :3], y[1, 0, 4:])) == 0).all()
    y, _ = idx.norm_rotary(q, None, eps=0.0)
    clean()
    assert torch.isnan(y[0, 0]).all() and torch.isfinite(y[2:]).all()

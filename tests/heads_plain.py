"""Plain 64-bit forms of the normalised and rotated heads and of the 4-bit cache, in numpy.  They share
no code with the package.

A four-bit code is decoded from the format (sign, two exponent bits with bias 1, one mantissa bit) and
rounded to by its sorted list of values.
"""
from __future__ import annotations

import numpy as np


def _decode(code):
    e, m = (code >> 1) & 3, code & 1
    v = m * 0.5 if e == 0 else (1 + m * 0.5) * 2.0 ** (e - 1)
    return -v if code & 8 else v


E2M1 = np.array([_decode(c) for c in range(16)])
_POS = E2M1[:8]  # 0 .. 6, ascending
BORDERS = (_POS[1:] + _POS[:-1]) / 2


def codes_of(packed):
    """uint8 [..., n] -> codes [..., 2 n], the low half first."""
    p = np.asarray(packed)
    return np.stack((p & 15, p >> 4), -1).reshape(*p.shape[:-1], -1)


def values4(packed):
    return E2M1[codes_of(packed)]


def e2m1(x):
    """The nearest values, ties to the even code, past 6 to 6."""
    a = np.minimum(np.abs(np.asarray(x, dtype=np.float64)), 6.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, 7)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    return np.copysign(_POS[np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)], x)


def ue8m0(byte):
    b = np.asarray(byte, dtype=np.float64)
    return np.where(b == 255, np.nan, 2.0 ** (b - 127))


def keys4(packed, scales):
    """Keys' numbers from codes [..., D/2] and bytes [..., D/32]."""
    v = values4(packed)
    return v * np.repeat(ue8m0(scales), 32, axis=-1)


def finite_max(x, axis):
    a = np.abs(x)
    return np.max(np.where(np.isfinite(a), a, 0.0), axis=axis)


def key_scale(amax):
    """The least exponent of -100 or more with amax <= 6 * 2^e."""
    e = -100
    while amax > 6.0 * 2.0 ** e:
        e += 1
    return e


def rotate_axes(x, positions, pair_axis, table, interleaved, offset, back=False):
    """x [T, H, D] float64, positions [A][T], table [P, r/2, 2]: pair i turned by its own axis'
    position; positions out of the table leave their pairs."""
    y = x.copy()
    half = table.shape[1]
    for t in range(x.shape[0]):
        for i in range(half):
            p = int(positions[pair_axis[i]][t])
            if not 0 <= p < table.shape[0]:
                continue
            a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + half + i)
            c, s = float(table[p, i, 0]), float(table[p, i, 1])
            s = -s if back else s
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


def rotate_f32(x, positions, table, interleaved, offset):
    """x [T, H, D] float32, turned in float32: products rounded, then their sum (what a rounding to four
    bits is defined on)."""
    y = x.copy()
    half = table.shape[1]
    with np.errstate(invalid="ignore"):
        for t, p in enumerate(positions):
            if not 0 <= p < table.shape[0]:
                continue
            c, s = table[p, :, 0], table[p, :, 1]
            a = offset + (2 * np.arange(half) if interleaved else np.arange(half))
            b = a + (1 if interleaved else half)
            y[t][:, a] = x[t][:, a] * c - x[t][:, b] * s
            y[t][:, b] = x[t][:, b] * c + x[t][:, a] * s
    return y


def norm(x, w, eps):
    """x [T, H, D] over its heads' root mean squares, times w."""
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def norm_gradients(x, w, eps, g):
    """(dx, dw) for the gradient g of norm(x, w, eps)."""
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    gw = g * w
    return r * gw - x * r ** 3 * (gw * x).mean(-1, keepdims=True), (g * x * r).sum((0, 1))

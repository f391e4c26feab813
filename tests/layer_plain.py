"""Plain 64-bit forms of the operators around the indexer, in numpy, one element or row at a time
where that is the shortest way to say it.  They share no code with the package.

e4m3 bytes are decoded from the format (sign, 4 exponent bits with bias 7, 3 mantissa bits, all
ones = NaN) and rounded to by searching the sorted list of its values.
"""
from __future__ import annotations

import math

import numpy as np


def _decode(byte):
    s, e, m = byte >> 7, (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if s else v


E4M3 = np.array([_decode(b) for b in range(256)])
_POS = E4M3[:127]  # 0 .. 448, ascending


def e4m3(x):
    """To nearest even, values past 448 to 448, NaN to NaN: the values, in float64."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), np.nan, np.copysign(_POS[pick], x))


def rotate(x, positions, table, interleaved, offset):
    """x [T, H, D] float64, table [P, r/2, 2] -> float64; positions out of the table stay."""
    y = x.copy()
    half = table.shape[1]
    for t, p in enumerate(positions):
        if not 0 <= p < table.shape[0]:
            continue
        for i in range(half):
            a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + half + i)
            c, s = float(table[p, i, 0]), float(table[p, i, 1])
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


def placement(seq_lens, new):
    """(request, position) of each new token, request by request."""
    return [(b, n - k + i) for b, (n, k) in enumerate(zip(seq_lens, new)) for i in range(k)]


def finite_max(x):
    a = np.abs(x)
    return float(np.max(np.where(np.isfinite(a), a, 0.0), initial=0.0))


def row_scale(x):
    return max(finite_max(x), 2.0 ** -100) / 448.0


def block_scale(amax):
    e = -100
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, pool, scales, table, seq_lens, new, block):
    """x [T, H, D] float64 (rotated) into pool float64 [N, H, block, D] (values) and scales
    [N, H], in place."""
    places = placement(seq_lens, new)
    done = set()
    for b, p in places:
        if p < 0 or (b, p // block) in done:
            continue
        j = p // block
        done.add((b, j))
        rows = [t for t, (bb, q) in enumerate(places) if bb == b and q >= 0 and q // block == j]
        at = [places[t][1] % block for t in rows]
        page = int(table[b][j])
        for h in range(pool.shape[1]):
            s = block_scale(finite_max(x[rows, h]))
            if at[0] > 0:
                was = float(scales[page, h])
                if s > was:
                    pool[page, h, :at[0]] = e4m3(pool[page, h, :at[0]] * (was / s))
                else:
                    s = was
            pool[page, h, at] = e4m3(x[rows, h] / s)
            scales[page, h] = s


def attention(q, k, v, ks, vs, table, seq_lens, block, scale, picked=None):
    """q [B, n, H, D]; k, v float64 values [N, Hkv, block, D].  picked: None, or a list of
    positions for each row.  Returns (out, lse, sum_p softmax_p |vs v_p|, the rows' positions)."""
    B, n, H, D = q.shape
    G = H // k.shape[1]
    out, mag = np.zeros((B, n, H, D)), np.zeros((B, n, H, D))
    lse = np.full((B, n, H), -np.inf)
    seen = []
    for b in range(B):
        for t in range(n):
            extent = max(0, int(seq_lens[b]) - n + t + 1)
            pos = list(range(extent)) if picked is None else \
                [p for p in picked[b * n + t] if 0 <= p < extent]
            seen.append(pos)
            if not pos:
                continue
            pos = np.array(pos)
            page = np.asarray(table[b])[pos // block]
            for g in range(k.shape[1]):
                kk = k[page, g, pos % block] * ks[page, g][:, None]
                vv = v[page, g, pos % block] * vs[page, g][:, None]
                for h in range(g * G, (g + 1) * G):
                    z = scale * (kk @ q[b, t, h])
                    m = z.max()
                    e = np.exp(z - m)
                    w = e / e.sum()
                    out[b, t, h], mag[b, t, h] = w @ vv, w @ np.abs(vv)
                    lse[b, t, h] = m + math.log(e.sum())
    return out, lse, mag, seen

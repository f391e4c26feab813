"""The 4-bit K/V cache: its writer, its reader and the attention over it, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import heads_plain as plain4
import layer_plain as plain
import paged_fp8_mqa_gb300 as idx

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
FLOOR = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


def dev():
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().cpu().double().numpy()


def u8(t):
    return t.detach().cpu().numpy()


def clean(bits=0):
    torch.cuda.synchronize()
    assert idx.device_status(clear=True) == bits


def pages_for(lens, bs, g, spare=2):
    need = [-(-n // bs) for n in lens]
    perm = torch.randperm(sum(need) + spare, generator=g).tolist()
    rows, at = [], 0
    for n in need:
        rows.append(perm[at:at + n])
        at += n
    width = max(need + [1])
    return [r + [10 ** 6] * (width - len(r)) for r in rows], sum(need) + spare


def empty_cache(blocks, H, bs, D, g):
    """Pools that hold something already."""
    kp, vp = (torch.randint(256, (blocks, H, bs, D // 2), generator=g, dtype=torch.uint8) for _ in range(2))
    ks = torch.randint(120, 130, (blocks, H, bs, D // 32), generator=g, dtype=torch.uint8)
    vs = torch.rand(blocks, H, bs, generator=g) + 0.1
    return [t.to(dev()) for t in (kp, vp, ks, vs)]


# ---- the writer and the reader -------------------------------------------------------------------

CASES = [  # request lengths, their new tokens
    ([1], [1]),
    ([5, 70, 64, 33], [5, 3, 64, 1]),
    ([130, 1, 200, 0, 65], [130, 1, 7, 0, 65]),
    ([40, 41, 42], [2, 2, 2]),
    ([1, 300], [4, 4]),  # shorter than its new tokens
]


def check_rows(x, k_codes, k_bytes, v, v_codes, v_scale):
    """One token's rows x (turned, float32) and v (float64) [H, D] against what was written."""
    for h in range(x.shape[0]):
        for j in range(x.shape[1] // 32):
            part = x[h, 32 * j:32 * j + 32].astype(np.float64)
            if np.isnan(part).any():
                assert k_bytes[h, j] == 255
                continue
            e = plain4.key_scale(plain4.finite_max(part, -1))
            assert k_bytes[h, j] == e + 127
            assert (plain4.values4(k_codes[h, 16 * j:16 * j + 16]) == plain4.e2m1(part / 2.0 ** e)).all()
        if np.isnan(v[h]).any():
            assert np.isnan(v_scale[h])
            continue
        most = max(plain4.finite_max(v[h], -1), 2.0 ** -96)
        assert v_scale[h] == np.float32(np.float32(most) / np.float32(6))
        y = np.clip(v[h], -most, most) * 6 / most
        got = plain4.values4(v_codes[h])
        # Quotients of 16-bit elements round alike in 32 bits and in 64; of float32 ones not within
        # 2^-22 of the border between two codes.
        near = (np.abs(np.abs(y)[:, None] - plain4.BORDERS) <= 2.0 ** -22 * np.abs(y)[:, None]).any(-1)
        exact = v.dtype != np.float32
        assert ((got == plain4.e2m1(y)) | (near & (not exact))).all()


@pytest.mark.parametrize("lens,new", CASES)
@pytest.mark.parametrize("D,bs,H,rot,offset,interleaved,name", [
    (128, 64, 2, 64, 0, False, "bf16"),
    (128, 32, 3, 128, 0, True, "f16"),
    (64, 128, 1, 32, 32, False, "bf16"),
    (64, 32, 8, 20, 6, True, "f32"),      # pairs that do not fill pieces
    (128, 64, 5, 0, 0, False, "f32"),
])
@pytest.mark.parametrize("layout", ["plain", "strided", "odd"])
def test_append_and_read(lens, new, D, bs, H, rot, offset, interleaved, name, layout):
    clean()
    g = gen(sum(lens) + D)
    rows, blocks = pages_for(lens, bs, g)
    cache = empty_cache(blocks, H, bs, D, g)
    was = [t.clone() for t in cache]
    T = sum(new)
    ragged = len(set(new)) > 1
    pad = 3 if ragged else 0  # (rows of no request behind the last)
    gap = dict(plain=0, strided=8, odd=3)[layout]
    k, v = (torch.randn(T + pad, H + (gap > 0), D + gap, generator=g).to(DTYPES[name]).to(dev())[:, :H, :D] for _ in range(2))
    k[:, :, D // 2] *= 50
    k[0, 0, :32] = 0
    v[-1 - pad, 0] = 0
    table = idx.rotary_table(max(lens) + 1, rot) if rot else None
    bt = torch.tensor(rows, dtype=torch.int32).to(dev())
    seq = torch.tensor(lens, dtype=torch.int32).to(dev())
    starts = torch.tensor([0, *np.cumsum(new)], dtype=torch.int32).to(dev()) if ragged else None
    how = dict(token_starts=starts, table=table, interleaved=interleaved, rot_offset=offset)
    idx.kv_append_fp4(k, v, *cache, bt, seq, **how)
    clean()
    place = [(b, m - n + i) for b, (m, n) in enumerate(zip(lens, new)) for i in range(n)]
    x = k.float().cpu().numpy()[:T]
    if rot:
        x = plain4.rotate_f32(x, [p for _, p in place], table.cpu().numpy(), interleaved, offset)
    vv = v.float().cpu().numpy()[:T]
    vv = vv if name == "f32" else vv.astype(np.float64)
    kp, vp, ks, vs = (u8(t) for t in cache)
    touched = np.zeros((blocks, bs), dtype=bool)
    for t, (b, p) in enumerate(place):
        if p < 0:
            continue
        page, at = rows[b][p // bs], p % bs
        touched[page, at] = True
        check_rows(x[t], kp[page, :, at], ks[page, :, at], vv[t], vp[page, :, at], vs[page, :, at])
    for now, then in zip(cache, was):  # everything else as it was
        assert (u8(now.transpose(1, 2))[~touched] == u8(then.transpose(1, 2))[~touched]).all()
    # Read back: the values, rounded once; rows of no request are zeros, or stay.
    for back in ("bf16", "f16", "f32"):
        ko, vo = idx.kv_read_fp4(*cache, bt, seq, starts, tokens=T + pad, dtype=DTYPES[back])
        clean()
        mine = [torch.full((T + pad, H + 1, D + gap), 7.0, dtype=DTYPES[back], device=dev())[:, :H, :D] for _ in range(2)]
        idx.kv_read_fp4(*cache, bt, seq, starts, tokens=T + pad, k_out=mine[0], v_out=mine[1])
        for t in range(T + pad):
            live = t < T and place[t][1] >= 0
            for got, given, codes, is_k in ((ko, mine[0], kp, True), (vo, mine[1], vp, False)):
                if not live:
                    assert (got[t] == 0).all() and (given[t] == 7).all()
                    continue
                page, at = rows[place[t][0]][place[t][1] // bs], place[t][1] % bs
                if is_k:
                    want = plain4.keys4(codes[page, :, at], ks[page, :, at])
                else:  # (one rounding to float32 before the type's)
                    want = (plain4.values4(codes[page, :, at]) * vs[page, :, at][:, None].astype(np.float64)).astype(np.float32)
                want = torch.tensor(want).to(DTYPES[back])
                assert torch.equal(got[t].cpu(), want) and torch.equal(given[t].cpu(), want)


def test_append_with_what_is_not_finite():
    """Infinities are held at the largest code, a NaN makes its scale NaN; the largest and least values."""
    for name in ("bf16", "f32"):
        D, bs = 64, 32
        cache = empty_cache(1, 1, bs, D, gen(0))
        k, v = (torch.randn(5, 1, D, generator=gen(i)).to(DTYPES[name]).to(dev()) for i in (1, 2))
        top = torch.finfo(DTYPES[name]).max
        k[0, 0, 3], v[0, 0, 3] = math.inf, -math.inf
        k[1, 0, 40], v[1, 0, 40] = math.nan, math.nan
        k[2, 0, 1], v[2, 0, 1] = top, -top
        k[3] *= 1e-36
        v[3] *= 1e-36
        k[4, 0, :32], v[4] = math.inf, math.inf
        idx.kv_append_fp4(k, v, *cache, torch.zeros(1, 1, dtype=torch.int32, device=dev()),
                          torch.tensor([5], dtype=torch.int32, device=dev()))
        clean()
        kp, vp, ks, vs = (u8(t)[0] for t in cache)
        X, V = k.float().cpu().numpy(), v.float().cpu().numpy()
        for t in range(5):
            if t == 4:
                assert (plain4.values4(kp[:, t])[0, :32] == 6).all() and ks[0, t, 0] == 27
                assert (plain4.values4(vp[:, t]) == 6).all()
                continue
            check_rows(X[t], kp[:, t], ks[:, t], V[t] if name == "f32" else V[t].astype(np.float64), vp[:, t], vs[:, t])
        # The values that a NaN's neighbours hold are read as NaN, the others as they are.
        ko, vo = idx.kv_read_fp4(*cache, torch.zeros(1, 1, dtype=torch.int32, device=dev()),
                                 torch.tensor([5], dtype=torch.int32, device=dev()), tokens=5, dtype=torch.float32)
        assert torch.isnan(ko[1, 0, 32:]).all() and not torch.isnan(ko[1, 0, :32]).any()
        assert torch.isnan(vo[1]).all() and not torch.isnan(vo[0]).any()


def test_ties_go_to_the_even_code():
    """Elements exactly between two codes, of scales that are no powers of two."""
    D = 64
    for top in (6.0, 9.0, 5.25, 0.046875):
        v = torch.zeros(1, 1, D)
        v[0, 0, 0] = top
        ties = torch.tensor(plain4.BORDERS) * top / 6
        v[0, 0, 1:8], v[0, 0, 8:15] = ties, -ties
        v = v.bfloat16()
        good = (v[0, 0, 1:8].double() * 6 == torch.tensor(plain4.BORDERS) * top).numpy()
        assert good.any()
        cache = empty_cache(1, 1, 32, D, gen(0))
        idx.kv_append_fp4(v.to(dev()), v.to(dev()), *cache, torch.zeros(1, 1, dtype=torch.int32, device=dev()),
                          torch.ones(1, dtype=torch.int32, device=dev()))
        got = plain4.values4(u8(cache[1])[0, 0, 0])
        want = plain4.e2m1(plain4.BORDERS)
        assert (got[1:8] == want)[good].all() and (got[8:15] == -want)[good].all()


def test_writers_and_readers_skip_and_flag():
    """A page outside the pool, a table too narrow, a position past the rotary table."""
    g = gen(3)
    cache = empty_cache(4, 1, 32, 64, g)
    was = [t.clone() for t in cache]
    k, v = (torch.randn(3, 1, 64, generator=g).bfloat16().to(dev()) for _ in range(2))
    bt = torch.tensor([[0, 4], [-1, 1], [2, 3]], dtype=torch.int32, device=dev())
    seq = torch.tensor([40, 10, 70], dtype=torch.int32, device=dev())
    clean()
    idx.kv_append_fp4(k, v, *cache, bt, seq)
    clean(idx.IDX_DEV_BAD_PAGE)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, was))
    ko, vo = idx.kv_read_fp4(*cache, bt, seq, tokens=3)
    clean(idx.IDX_DEV_BAD_PAGE)
    assert (ko == 0).all() and (vo == 0).all()
    table = idx.rotary_table(5, 32)
    idx.kv_append_fp4(k[:1], v[:1], *cache, bt[2:], seq[2:] - 10, table=table)
    clean(idx.IDX_DEV_BAD_POSITION)
    check_rows(k[0].float().cpu().numpy(), u8(cache[0])[3, :, 27], u8(cache[2])[3, :, 27],
               f64(v[0]), u8(cache[1])[3, :, 27], u8(cache[3])[3, :, 27])


def test_long_runs_equal_their_parts():
    """Some thousands of tokens at once (several rows a warp) and in small calls: the same bytes."""
    g = gen(9)
    H, D, bs, lens = 4, 128, 64, [2900, 1501, 1]
    rows, blocks = pages_for(lens, bs, g)
    bt = torch.tensor(rows, dtype=torch.int32).to(dev())
    k, v = (torch.randn(sum(lens), H, D, generator=g).bfloat16().to(dev()) for _ in range(2))
    table = idx.rotary_table(3000, 64)
    whole, parts = empty_cache(blocks, H, bs, D, gen(1)), empty_cache(blocks, H, bs, D, gen(1))
    starts = torch.tensor([0, 2900, 4401, 4402], dtype=torch.int32).to(dev())
    idx.kv_append_fp4(k, v, *whole, bt, torch.tensor(lens, dtype=torch.int32).to(dev()), token_starts=starts, table=table)
    for b, n in enumerate(lens):
        for at in range(0, n, 700):
            m = min(700, n - at)
            idx.kv_append_fp4(k[starts[b] + at:starts[b] + at + m], v[starts[b] + at:starts[b] + at + m], *parts,
                              bt[b:b + 1], torch.tensor([at + m], dtype=torch.int32).to(dev()), table=table)
    clean()
    assert all(torch.equal(a, b) for a, b in zip(whole, parts))
    back = idx.kv_read_fp4(*whole, bt, torch.tensor(lens, dtype=torch.int32).to(dev()), starts, tokens=sum(lens))
    one = idx.kv_read_fp4(*whole, bt[1:2], torch.tensor([1501], dtype=torch.int32).to(dev()), tokens=200)
    assert torch.equal(back[0][2900 + 1301:4401], one[0]) and torch.equal(back[1][2900 + 1301:4401], one[1])


# ---- attention -----------------------------------------------------------------------------------

def attention_case(lens, n, H, Hkv, D, bs, name, seed, poison=True, qmag=1.0):
    """Inputs whose unseen positions and unused pages have NaN scales."""
    g = gen(seed)
    rows, blocks = pages_for(lens, bs, g)
    k, v = (torch.randint(256, (blocks, Hkv, bs, D // 2), generator=g, dtype=torch.uint8) for _ in range(2))
    ks = torch.randint(122, 127, (blocks, Hkv, bs, D // 32), generator=g, dtype=torch.uint8)
    vs = torch.rand(blocks, Hkv, bs, generator=g) * 0.4 + 0.1
    if poison:
        used = torch.zeros(blocks, bs, dtype=torch.bool)
        for b, m in enumerate(lens):
            for p in range(m):
                used[rows[b][p // bs], p % bs] = True
        ks.permute(0, 2, 1, 3)[~used] = 0xFF
        vs.permute(0, 2, 1)[~used] = math.nan
    q = (torch.randn(len(lens), n, H + 1, D + 8, generator=g) * qmag).to(DTYPES[name])
    return dict(q=q.to(dev())[:, :, 1:, :D], k=k.to(dev()), v=v.to(dev()), ks=ks.to(dev()), vs=vs.to(dev()),
                bt=torch.tensor([r + [10 ** 6] for r in rows], dtype=torch.int32).to(dev())[:, :-1],
                seq=torch.tensor([[m, -1] for m in lens], dtype=torch.int32).to(dev())[:, 0],
                rows=rows, lens=lens, bs=bs, name=name)


def run_attention(c, **more):
    B, n, H, _ = c["q"].shape
    lse = torch.full((B, n, H), math.nan, device=dev())
    out = idx.attention_fp4(c["q"], c["k"], c["v"], c["ks"], c["vs"], c["bt"], c["seq"], lse=lse, **more)
    torch.cuda.synchronize()
    return out, lse


def check_attention(c, out, lse, picked=None, scale=None):
    """Tolerance.  A query element is exact or held to 2^-31 of its row's largest, products are exact,
    sums are float32 (D / 32 steps a part, and the tensor core's own alignment, 2^-22 of a step's largest
    term): the scores are off by dz at most.  A weight is held to 2^-10 of itself (float16 2^-14) or
    2^-34 of the largest; the logarithm of a value scale, added to the score, and the base-2 exponential
    have 2^-20 between them.  The output is rounded once."""
    name, D = c["name"], c["q"].shape[3]
    scale = D ** -0.5 if scale is None else scale
    q = f64(c["q"])
    k = plain4.keys4(u8(c["k"]), u8(c["ks"]))
    v = plain4.values4(u8(c["v"])) * f64(c["vs"])[..., None]
    one = np.ones(k.shape[:2])
    ref, ref_lse, mag, seen = plain.attention(q, k, v, one, one, c["rows"], c["lens"], c["bs"], scale, picked)
    B, n, H, _ = q.shape
    G = H // k.shape[1]
    got, got_lse = f64(out), f64(lse)
    w_rel = (2.0 ** -10 if name == "bf16" else 2.0 ** -14) + 2.0 ** -18
    for b in range(B):
        for t in range(n):
            pos = np.array(seen[b * n + t], dtype=int)
            if not pos.size:
                assert (got[b, t] == 0).all() and (got_lse[b, t] == -np.inf).all()
                continue
            page = np.asarray(c["rows"][b])[pos // c["bs"]]
            for h in range(H):
                kk = k[page, h // G, pos % c["bs"]]
                vv = np.abs(v[page, h // G, pos % c["bs"]])
                qq = q[b, t, h]
                z = scale * (kk @ qq)
                dz = abs(scale) * np.max(2.0 ** -30 * np.abs(qq).max() * np.abs(kk).sum(1) + 2.0 ** -19 * (np.abs(kk) @ np.abs(qq)))
                dz += 2.0 ** -21 * np.abs(z).max() + 2.0 ** -20
                u = np.exp(z - z.max()) * np.maximum(f64(c["vs"])[page, h // G, pos % c["bs"]], 0)
                low = 2.0 ** -33 * u.max() * np.abs(plain4.values4(u8(c["v"])[page, h // G, pos % c["bs"]])).sum(0) / np.exp(z - z.max()).sum()
                lim = (2 * dz + w_rel + len(pos) * 2.0 ** -24) * mag[b, t, h] + low
                lim = lim + HALF_ULP[name] * (np.abs(ref[b, t, h]) + lim) + FLOOR[name]
                err = np.abs(got[b, t, h] - ref[b, t, h])
                assert (err <= lim).all(), (b, t, h, float(np.max(err / lim)))
                assert abs(got_lse[b, t, h] - ref_lse[b, t, h]) <= dz + 2.0 ** -20 * (1 + abs(ref_lse[b, t, h])) + len(pos) * 2.0 ** -24


SHAPES = [  # H, Hkv, D, block, dtype
    (8, 8, 128, 64, "bf16"),     # a head of its own for each query head
    (16, 2, 128, 64, "bf16"),
    (6, 2, 64, 32, "f16"),       # groups of three
    (8, 1, 64, 64, "bf16"),
    (64, 1, 128, 128, "f16"),
    (70, 2, 64, 64, "bf16"),     # groups of 35
    (13, 1, 128, 32, "f16"),
    (28, 1, 64, 128, "bf16"),
    (130, 1, 128, 64, "bf16"),   # more rows than one tile of queries holds
]
LENS = [300, 0, 1, 3, 31, 33, 64, 127, 128, 129, 257, 1000]


@pytest.mark.parametrize("H,Hkv,D,bs,name", SHAPES)
@pytest.mark.parametrize("n", [1, 2, 4])
def test_attention_over_every_position(H, Hkv, D, bs, name, n):
    clean()
    c = attention_case(LENS, n, H, Hkv, D, bs, name, H + n)
    out, lse = run_attention(c)
    clean()
    check_attention(c, out, lse)
    again, _ = run_attention(c)
    assert torch.equal(out, again)  # the same bits each time


@pytest.mark.parametrize("D,num_sms", [(128, 1), (128, 3), (128, 40), (64, 1), (64, 7)])
def test_attention_split_any_way(D, num_sms):
    """Few CTAs walk many requests each; many CTAs share one request."""
    for lens in (LENS, [5000], [5] * 70):
        c = attention_case(lens, 2, 16, 2, D, 32, "bf16", 17)
        out, lse = run_attention(c, num_sms=num_sms)
        check_attention(c, out, lse)
    clean()


def selections(c, top_k, g, extra=3):
    """Slots as the select leaves them, with positions no row can see among them."""
    B, n = c["q"].shape[:2]
    slots = 2 * top_k + 8
    cand = torch.randint(-2 ** 30, 2 ** 30, (B * n, slots, 2), generator=g, dtype=torch.int32)
    ranges = torch.zeros(2, B * n, dtype=torch.int32)
    picked = []
    for r in range(B * n):
        extent = max(0, c["lens"][r // n] - n + r % n + 1)
        count = min(extent, top_k + extra * (r % 3))
        p = torch.randperm(extent, generator=g)[:count].tolist() if extent else []
        if count > 4:
            p[2] = p[0]                 # twice the same
            p[1] = extent + 1 + r       # past the extent
            p[3] = -1 - r
        lo = top_k - min(r % 3, count)
        cand[r, lo:lo + count, 0] = torch.tensor(p, dtype=torch.int32)
        ranges[0, r], ranges[1, r] = lo, lo + count
        picked.append(p)
    return cand.to(dev()), ranges.to(dev()), picked


@pytest.mark.parametrize("H,Hkv,D,bs,name", SHAPES)
@pytest.mark.parametrize("n,top_k", [(1, 64), (2, 200), (4, 5)])
def test_attention_over_the_selected_positions(H, Hkv, D, bs, name, n, top_k):
    clean()
    c = attention_case(LENS, n, H, Hkv, D, bs, name, H + n + top_k)
    cand, ranges, picked = selections(c, top_k, gen(n))
    out, lse = run_attention(c, candidates=cand, ranges=ranges)
    clean()
    check_attention(c, out, lse, picked)


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_attention_with_large_scores(name):
    """Scores of a few hundred: one position carries a row, and others' weights vanish."""
    c = attention_case([5, 700, 130], 1, 16, 2, 128, 64, name, 23, qmag=30.0)
    for scale in (None, 0.0, -0.05):
        out, lse = run_attention(c, softmax_scale=scale)
        check_attention(c, out, lse, scale=scale)
    clean()


@pytest.mark.parametrize("D", [64, 128])
def test_attention_with_scales_far_apart(D):
    """Keys' groups 2^40 apart, value scales 2^24, a value scale of 0 and a negative one; an outlier in the
    queries that meets no key's element; zero queries."""
    c = attention_case([256, 300], 1, 8, 1, D, 32, "bf16", 29)
    g = gen(2)
    c["ks"][..., 0] = torch.randint(86, 90, c["ks"].shape[:3], generator=g).to(torch.uint8).to(dev())
    c["k"][..., 16:20] = 0  # (elements 32 .. 39)
    c["q"] = c["q"].clone()
    c["q"][:, :, :, 33] = 2.0 ** 17
    c["q"][1, 0, 3] = 0.0
    c["vs"] = c["vs"] * 2.0 ** (-12.0 * torch.randint(3, c["vs"].shape, generator=g).to(dev()))
    c["vs"][c["rows"][0][0], :, 3] = 0.0
    out, lse = run_attention(c)
    check_attention(c, out, lse)
    clean()


def test_attention_with_negative_and_zero_value_scales():
    c = attention_case([300, 64, 129], 1, 8, 1, 128, 64, "bf16", 53)
    plain_out, plain_lse = run_attention(c)
    flip = (torch.arange(c["vs"].numel(), device=dev()) % 3 == 0).view_as(c["vs"])
    neg = dict(c, vs=torch.where(flip, -c["vs"], c["vs"]))
    out, lse = run_attention(neg)
    # A negative scale is its rows' codes with the other sign.
    same = dict(c, v=torch.where(flip[..., None], c["v"] ^ 0x88, c["v"]))
    want, want_lse = run_attention(same)
    assert torch.equal(lse, want_lse)
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
    for page in c["rows"][2][:3]:
        c["vs"][page] = 0.0
    out, lse = run_attention(c)
    assert (out[2] == 0).all() and torch.equal(out[:2], plain_out[:2]) and not torch.isnan(lse).any()
    clean()


@pytest.mark.parametrize("D,picked", [(128, False), (64, False), (128, True)])
@pytest.mark.parametrize("what", ["key", "value", "infinite value"])
def test_a_scale_that_is_not_finite_reaches_the_rows_that_see_it(D, picked, what):
    n, lens = 4, [130, 64, 6]
    c = attention_case(lens, n, 8, 2, D, 64, "bf16", 31)
    more = {}
    if picked:
        cand = torch.arange(160, dtype=torch.int32).repeat(12, 1)[..., None].repeat(1, 1, 2).to(dev()).contiguous()
        ranges = torch.tensor([[0] * 12, [max(0, lens[r // 4] - 3 + r % 4) for r in range(12)]], dtype=torch.int32).to(dev())
        more = dict(candidates=cand, ranges=ranges)
    base, base_lse = run_attention(c, **more)
    for b, m in enumerate(lens):
        p = m - 2  # seen by slots 2 and 3
        page, at = c["rows"][b][p // 64], p % 64
        if what == "key":
            c["ks"][page, 1, at, 1] = 0xFF
        else:
            c["vs"][page, 1, at] = math.nan if what == "value" else math.inf
    out, lse = run_attention(c, **more)
    clean()
    assert torch.equal(out[:, :2], base[:, :2]) and torch.equal(lse[:, :2], base_lse[:, :2])
    assert torch.equal(out[:, 2:, :4], base[:, 2:, :4])
    assert torch.isnan(out[:, 2:, 4:]).all() and torch.isnan(lse[:, 2:, 4:]).all()


def test_attention_flags_bad_pages():
    """A block id outside the pool and a table too narrow: those positions are passed over."""
    for D in (64, 128):
        c = attention_case([200, 130], 1, 8, 2, D, 32, "bf16", 37)
        c["bt"][0, 2] = 10 ** 6
        c["bt"][1, 0] = -1
        out, lse = run_attention(c)
        clean(idx.IDX_DEV_BAD_PAGE)
        check_attention(c, out, lse, [[p for p in range(200) if p // 32 != 2], list(range(32, 130))])
        c["bt"] = torch.tensor(c["rows"], dtype=torch.int32).to(dev())[:, :3]
        out, lse = run_attention(c)
        clean(idx.IDX_DEV_BAD_PAGE)
        check_attention(c, out, lse, [list(range(96)), list(range(96))])
        cand, ranges, picked = selections(c, 50, gen(2))
        out, lse = run_attention(c, candidates=cand, ranges=ranges)
        clean(idx.IDX_DEV_BAD_PAGE)
        check_attention(c, out, lse, [[p for p in row if p < 96] for row in picked])


@pytest.mark.parametrize("H,bs,name,n", [(8, 32, "bf16", 1), (16, 64, "bf16", 1), (17, 128, "f16", 1),
                                         (9, 32, "bf16", 4), (32, 64, "bf16", 2), (16, 32, "f16", 1)])
def test_attention_where_two_tokens_share_a_row(H, bs, name, n):
    """head_dim 64: lengths that end at the first and the second token of a pair and around a tile of 256, one
    chunk of 16 rows and several, a page of the middle that is not there."""
    clean()
    c = attention_case([255, 256, 2, 1, 511, 512, 513], n, H, 1, 64, bs, name, 90 + H)
    check_attention(c, *run_attention(c))
    clean()
    c["bt"][5, 1] = -1
    out, lse = run_attention(c)
    clean(idx.IDX_DEV_BAD_PAGE)
    there = [[p for p in range(m - n + t + 1) if b != 5 or p // bs != 1] for b, m in enumerate(c["lens"])
             for t in range(n)]
    check_attention(c, out, lse, there)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_and_reader_past_32_bits_of_a_pool(D):
    bs = 128
    blocks = (1 << 32) // (bs * D // 2) + 40  # (2^32 bytes of codes; rows stay below 2^31)
    c = attention_case([300, 90], 1, 4, 1, D, bs, "bf16", 41)
    first = blocks - c["k"].shape[0]
    for name in ("k", "v", "ks", "vs"):
        t = c[name]
        big = torch.zeros((blocks, *t.shape[1:]), dtype=t.dtype, device=dev())
        big[first:] = t
        c[name + "_big"] = big
    far = dict(c, bt=torch.where(c["bt"] < 10 ** 6, c["bt"] + first, c["bt"]),
               **{m: c[m + "_big"] for m in ("k", "v", "ks", "vs")})
    out, lse = run_attention(far)
    cand, ranges, picked = selections(c, 60, gen(2))
    some, some_lse = run_attention(far, candidates=cand, ranges=ranges)
    kv = idx.kv_read_fp4(far["k"], far["v"], far["ks"], far["vs"], far["bt"], far["seq"], tokens=180)
    clean()
    check_attention(c, out, lse)
    check_attention(c, some, some_lse, picked)
    near = idx.kv_read_fp4(c["k"], c["v"], c["ks"], c["vs"], c["bt"], c["seq"], tokens=180)
    assert all(torch.equal(a, b) for a, b in zip(kv, near))
    idx.kv_append_fp4(kv[0][:2], kv[1][:2], far["k"], far["v"], far["ks"], far["vs"], far["bt"], far["seq"])
    idx.kv_append_fp4(kv[0][:2], kv[1][:2], c["k"], c["v"], c["ks"], c["vs"], c["bt"], c["seq"])
    clean()
    assert torch.equal(far["k"][first:], c["k"]) and torch.equal(far["vs"][first:].view(torch.int32), c["vs"].view(torch.int32))


def test_on_another_stream_and_in_a_graph_with_two_workspaces():
    c = attention_case([700, 80, 0, 333], 1, 16, 2, 128, 64, "bf16", 43)
    want, _ = run_attention(c)
    args = c["q"], c["k"], c["v"], c["ks"], c["vs"], c["bt"], c["seq"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = idx.attention_fp4(*args, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    need = idx.idx_attention_workspace_bytes(4, 1, 16, 2, 128, 0)
    ws = torch.zeros(need, dtype=torch.uint8, device=dev())
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx.attention_fp4(*args, out=out, workspace=ws)
    for _ in range(3):
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    clean()


def test_a_decode_step_norms_appends_and_attends():
    """The operators together, as a layer uses them, against the same on dense tensors in 64 bits: prompts
    in, then steps of normalised and rotated queries and keys."""
    clean()
    H, Hkv, D, bs, most = 8, 2, 128, 64, 200
    g = gen(61)
    lens = [70, 1, 128]
    rows, blocks = pages_for([most] * 3, bs, g)
    bt = torch.tensor(rows, dtype=torch.int32).to(dev())
    cache = empty_cache(blocks, Hkv, bs, D, g)
    axes = idx.rotary_axes((16, 24, 24))
    table = idx.rotary_table(300, 128)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=g)).bfloat16().to(dev()) for _ in range(2))

    def step(T):
        qkv = torch.randn(T, H + 2 * Hkv, D, generator=g).bfloat16().to(dev())
        pos = torch.randint(300, (3, T), generator=g, dtype=torch.int32).to(dev())
        q, k = idx.norm_rotary(qkv[:, :H], qkv[:, H:H + Hkv], wq, wk, pos, table, axes=axes)
        return q, k, qkv[:, H + Hkv:]

    T = sum(lens)
    starts = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32).to(dev())
    seq = torch.tensor(lens, dtype=torch.int32).to(dev())
    _, k, v = step(T)
    idx.kv_append_fp4(k, v, *cache, bt, seq, token_starts=starts)
    for i in range(3):
        q, k, v = step(3)
        seq = seq + 1
        idx.kv_append_fp4(k, v, *cache, bt, seq)
    q = q.view(3, 1, H, D)
    lse = torch.empty(3, 1, H, device=dev())
    out = idx.attention_fp4(q, *cache, bt, seq, lse=lse)
    clean()
    kp, vp, ks, vs = cache
    c = dict(q=q, k=kp, v=vp, ks=ks, vs=vs, rows=rows, lens=seq.tolist(), bs=bs, name="bf16")
    check_attention(c, out, lse)
    # The last key is the step's, within its codes' half steps.
    kk, _ = idx.kv_read_fp4(*cache, bt, seq, tokens=3, dtype=torch.float32)
    scale = 2.0 ** torch.ceil(torch.log2(k.float().unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True) / 6))
    assert ((kk - k.float()).unflatten(-1, (-1, 32)).abs() <= scale).all()


def test_refusals_of_tensors():
    g = gen(1)
    cache = empty_cache(4, 2, 32, 64, g)
    kp, vp, ks, vs = cache
    x = torch.randn(3, 2, 64, generator=g).bfloat16().to(dev())
    bt = torch.zeros(3, 1, dtype=torch.int32, device=dev())
    seq = torch.ones(3, dtype=torch.int32, device=dev())
    starts = torch.zeros(1, dtype=torch.int32, device=dev())
    wide = torch.zeros(3, 1, 2, 64, dtype=torch.bfloat16, device=dev())
    for bad, error in (
            (lambda: idx.kv_append_fp4(x, x.half(), *cache, bt, seq), TypeError),
            (lambda: idx.kv_append_fp4(x, x, kp.float(), vp, ks, vs, bt, seq), TypeError),
            (lambda: idx.kv_append_fp4(x, x, kp, vp, ks[..., :1], vs, bt, seq), ValueError),
            (lambda: idx.kv_append_fp4(x, x, kp, vp, ks, vs[:, :1].expand(4, 2, 32), bt, seq), ValueError),
            (lambda: idx.kv_append_fp4(x, x, kp, vp[:3], ks, vs, bt, seq), ValueError),
            (lambda: idx.kv_append_fp4(x[:, :1], x[:, :1], *cache, bt, seq), ValueError),
            (lambda: idx.kv_append_fp4(x, x, *cache, bt[:1].expand(3, 1), seq), ValueError),
            (lambda: idx.kv_append_fp4(x[:2], x[:2], *cache, bt, seq), ValueError),
            (lambda: idx.kv_read_fp4(*cache, bt, seq, tokens=4), ValueError),
            (lambda: idx.kv_read_fp4(*cache, bt[:0], seq[:0], starts, tokens=4), ValueError),
            (lambda: idx.kv_read_fp4(*cache, bt, seq, tokens=3, dtype=torch.float64), TypeError),
            (lambda: idx.kv_read_fp4(*cache, bt, seq, tokens=3, k_out=x), ValueError),
            (lambda: idx.kv_read_fp4(*cache, bt, seq, tokens=3, k_out=x, v_out=x[:1].expand(3, 2, 64)), ValueError),
            (lambda: idx.attention_fp4(wide.float(), *cache, bt, seq), TypeError),
            (lambda: idx.attention_fp4(wide[..., :32], *cache, bt, seq), ValueError),
            (lambda: idx.attention_fp4(torch.cat([wide] * 5, 1), *cache, bt, seq), idx.IdxError),
            (lambda: idx.attention_fp4(wide[:, :, :1], *cache, bt, seq), idx.IdxError)):
        with pytest.raises(error):
            bad()
    torch.cuda.synchronize()
    k, v = idx.kv_read_fp4(*cache, bt, seq, torch.zeros(4, dtype=torch.int32, device=dev()), tokens=0)
    assert k.shape == (0, 2, 64) and v.dtype == torch.bfloat16


def codes_of_quotients(v, most):
    """Indices of the nearest values to 6 v / most, ties to the even code, by exact fractions."""
    from fractions import Fraction
    values = [Fraction(float(x)) for x in plain4.E2M1[:8]]
    out = []
    for x in v:
        y = min(abs(6 * Fraction(float(x)) / Fraction(float(most))), 6)
        i = min(range(8), key=lambda c: (abs(values[c] - y), c % 2))
        out.append(8 + i if x < 0 else i)
    return out


@pytest.mark.parametrize("layout", ["plain", "odd"])
@pytest.mark.parametrize("D,shift", [(64, 0), (128, -118), (64, 103)])
def test_float32_values_next_to_a_border(D, shift, layout):
    """Float32 elements whose quotient lies on a border between two codes, or within 2^-21 of it, where a
    quotient rounded to float32 would lie on it: the code is the exact quotient's."""
    g = np.random.default_rng(D + shift)
    rows = []
    for _ in range(200):
        most = int(g.integers(2 ** 23, 2 ** 24)) // 12 * 12 + int(g.integers(2)) * int(g.integers(12))
        most = min(max(most, 2 ** 23), 2 ** 24 - 1)
        row = [float(most)]
        for border in plain4.BORDERS:
            at = np.float32(border * most / 6)
            row += [np.nextafter(at, np.float32(0)), at, -at, np.nextafter(at, np.float32(2 ** 25))]
        rows.append(row + [0.0] * (D - len(row)))
    # (One that rounds to a tie both in 6 v and in the quotient.)
    rows[0][:2] = [13421820.0, 5592425.0]
    v = torch.tensor(np.array(rows, dtype=np.float32) * np.float32(2.0 ** shift))[:, None]
    wide = torch.zeros(200, 1, D + 3)
    wide[:, :, :D] = v
    given = v.to(dev()) if layout == "plain" else wide.to(dev())[:, :, :D]
    cache = empty_cache(7, 1, 32, D, gen(0))
    bt = torch.arange(7, dtype=torch.int32, device=dev())[None]
    clean()
    idx.kv_append_fp4(given, given, *cache, bt, torch.tensor([200], dtype=torch.int32, device=dev()))
    clean()
    got = plain4.codes_of(u8(cache[1]))[:, 0].reshape(-1, D)[:200]
    want = np.array([codes_of_quotients(row, max(row)) for row in v[:, 0].numpy()])
    # (A zero's code has no sign.)
    assert (np.where(v[:, 0].numpy() == 0, 0, got) == want).all()


@pytest.mark.parametrize("cache", ["fp8", "fp4"])
def test_attention_says_that_it_has_no_gradient(cache):
    """A query that requires a gradient (as norm_rotary leaves it in a model): the same result, and a backward
    pass through it is an error and not silence; a tangent is refused."""
    from torch.autograd import forward_ad
    H, D, bs = 4, 64, 32
    g = gen(3)
    bt, seq = torch.tensor([[1, 0]], dtype=torch.int32, device=dev()), torch.tensor([40], dtype=torch.int32, device=dev())
    if cache == "fp4":
        held, call = empty_cache(2, 1, bs, D, g), idx.attention_fp4
    else:
        held = [torch.randint(0x40, (2, 1, bs, D), generator=g, dtype=torch.uint8).to(dev()) for _ in range(2)]
        held += [torch.ones(2, 1, device=dev()) for _ in range(2)]
        call = idx.attention_fp8
    x = torch.randn(1, H, D, generator=g).bfloat16().to(dev())
    with torch.no_grad():
        q, _ = idx.norm_rotary(x, None)
        want = call(q[:, None], *held, bt, seq)
        assert not want.requires_grad
    leaf = x.clone().requires_grad_()
    q, _ = idx.norm_rotary(leaf, None)
    lse = torch.zeros(1, 1, H, device=dev())
    out = call(q[:, None], *held, bt, seq, lse=lse)
    assert torch.equal(out, want) and out.requires_grad and (lse != 0).all()
    with pytest.raises(NotImplementedError, match="attention_" + cache):
        out.float().sum().backward()
    assert leaf.grad is None
    with torch.no_grad():
        assert not call(q[:, None], *held, bt, seq).requires_grad
    given = torch.empty_like(want)
    assert call(q[:, None], *held, bt, seq, out=given) is given and not given.requires_grad
    assert torch.equal(given, want) and not call(q[:, None].detach(), *held, bt, seq).requires_grad
    with forward_ad.dual_level(), pytest.raises(NotImplementedError, match="attention_" + cache):
        call(forward_ad.make_dual(want, want), *held, bt, seq)
    clean()

"""Rotary positions, the writers of the two 8-bit pools and the attention over the K/V pool,
against their plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import layer_plain as plain
import oracle
import paged_fp8_mqa_gb300 as idx

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# Half a unit in the last place of each type (24, 11 and 8 bits of significand), relative to the
# least value of its binade, and the least subnormal's half.
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
FLOOR = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


def dev():
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().cpu().double().numpy()


def values8(t):
    """e4m3 bytes as the values they stand for, decoded by the plain table."""
    return plain.E4M3[t.detach().view(torch.uint8).cpu().numpy()]


def clean(bits=0):
    torch.cuda.synchronize()
    assert idx.device_status(clear=True) == bits


# ---- rotary --------------------------------------------------------------------------------------

def check_rotary(x, y, positions, table, interleaved, offset, name):
    ref = plain.rotate(f64(x), positions, f64(table), interleaved, offset)
    # Two products and a sum in float32 (three roundings of terms no larger than the pair's
    # magnitudes times |cos|, |sin|), then one rounding to the type.
    size = plain.rotate(np.abs(f64(x)), positions, np.abs(f64(table)) * [1, -1], interleaved, offset)
    mag = np.maximum(np.abs(f64(x)), np.abs(size))
    lim = HALF_ULP[name] * np.abs(ref) + FLOOR[name] + 3 * 2.0 ** -24 * 2 * mag.max(-1, keepdims=True)
    assert (np.abs(f64(y) - ref) <= lim).all(), np.max(np.abs(f64(y) - ref) - lim)


@pytest.mark.parametrize("T,H,D,rot,offset,interleaved,name", [
    (1, 1, 64, 64, 0, False, "bf16"),
    (7, 3, 128, 64, 64, True, "bf16"),
    (33, 5, 128, 128, 0, False, "f16"),
    (5, 64, 192, 64, 0, True, "f32"),
    (4, 2, 96, 48, 48, False, "bf16"),
    (3, 9, 80, 20, 30, False, "f16"),   # no vector path: rot / 2 = 10, offset 30
    (2, 2, 7, 2, 5, True, "f32"),       # odd rows
    (6, 1, 66, 66, 0, True, "bf16"),
])
@pytest.mark.parametrize("layout", ["plain", "strided", "in place"])
def test_rotary(T, H, D, rot, offset, interleaved, name, layout):
    clean()
    table = idx.rotary_table(600, rot)
    g = gen(T * 1000 + D)
    base = torch.randn(T, H + 1, D + 8, generator=g).to(DTYPES[name]).to(dev())
    x = base[:, 1:, :D] if layout == "strided" else base[:, :H, :D].contiguous()
    pos = torch.randint(600, (T,), generator=g, dtype=torch.int32)
    pos[0] = 599
    keep = x.clone()
    out = x if layout == "in place" else None
    y = idx.rotary(x, pos.to(dev()), table, interleaved=interleaved, rot_offset=offset, out=out)
    clean()
    assert (y.data_ptr() == x.data_ptr()) == (layout == "in place")
    if layout != "in place":
        assert torch.equal(x, keep)
    check_rotary(keep, y, pos.tolist(), table, interleaved, offset, name)


def test_rotary_gradient_is_the_inverse():
    """d/dx of sum(w * rotary(x)) by the inverse call, by the formula and by differences."""
    table = idx.rotary_table(100, 32, scaling="yarn", factor=4.0, original_positions=64)
    g = gen(3)
    x, w = (torch.randn(3, 2, 48, generator=g).to(dev()) for _ in range(2))
    pos = torch.tensor([0, 99, 41], dtype=torch.int32, device=dev())
    for interleaved in (False, True):
        call = lambda v: idx.rotary(v, pos, table, interleaved=interleaved, rot_offset=16)  # noqa: E731
        grad = f64(idx.rotary(w, pos, table, interleaved=interleaved, rot_offset=16, inverse=True))
        turned = f64(table) * [1, -1]
        ref = plain.rotate(f64(w), pos.tolist(), turned, interleaved, 16)
        assert np.abs(grad - ref).max() <= 6 * 2.0 ** -24 * np.abs(f64(w)).max() * 1.2
        # The map is linear: a difference over a step of 1 has the rounding of two outputs only.
        y0 = f64(call(x))
        for i in (0, 17, 30, 47):
            e = torch.zeros_like(x)
            e[1, 1, i] = 1.0
            diff = ((f64(call(x + e)) - y0) * f64(w)).sum()
            assert abs(diff - grad[1, 1, i]) <= 48 * 2.0 ** -22 * 8


def test_rotary_positions_outside_the_table():
    clean()
    table = idx.rotary_table(10, 16)
    x = torch.randn(4, 2, 16, generator=gen(1)).to(dev())
    pos = torch.tensor([3, -1, 10, 9], dtype=torch.int32)
    y = idx.rotary(x, pos.to(dev()), table)
    clean(idx.IDX_DEV_BAD_POSITION)
    assert torch.equal(y[1:3], x[1:3])
    check_rotary(x, y, pos.tolist(), table, False, 0, "f32")


@pytest.mark.parametrize("scaling,more", [
    ("none", {}), ("linear", dict(factor=8.0)), ("ntk", dict(factor=4.0)),
    ("yarn", dict(factor=16.0, original_positions=4096)),
])
def test_rotary_table_far_out(scaling, more):
    """The table's angles at far positions, against math.cos of the 64-bit angle; the frequencies
    themselves are checked on the CPU."""
    import ctypes
    rot, most = 64, 131072
    table = f64(idx.rotary_table(most, rot, scaling=scaling, **more))
    freq, mag = (ctypes.c_double * (rot // 2))(), ctypes.c_double()
    code = dict(none=0, linear=1, ntk=2, yarn=3)[scaling]
    assert idx.idx_rotary_frequencies(rot, 10000.0, code, more.get("factor", 1.0),
                                      more.get("original_positions", 0.0), 32.0, 1.0, freq,
                                      ctypes.byref(mag)) == 0
    for p in (0, 1, 4097, 99999, most - 1):
        for i in (0, 5, 31):
            c, s = mag.value * math.cos(p * freq[i]), mag.value * math.sin(p * freq[i])
            # One rounding to float32; the 64-bit sine is within 2e-16 * p of the angle's.
            assert abs(table[p, i, 0] - c) <= 2.0 ** -24 * 1.5 + 1e-10
            assert abs(table[p, i, 1] - s) <= 2.0 ** -24 * 1.5 + 1e-10


# ---- the writers ---------------------------------------------------------------------------------

def pages_for(lens, bs, g, spare=2):
    """Block tables (list of rows, padded with a page of nobody's) over a shuffled pool."""
    need = [-(-n // bs) for n in lens]
    width = max(max(need), 1)
    perm = torch.randperm(sum(need) + spare, generator=g).tolist()
    rows, at = [], 0
    for n in need:
        rows.append(perm[at:at + n] + [perm[-1]] * (width - n))
        at += n
    return rows, sum(need) + spare


CASES = [  # (seq_lens after the write, new tokens of each)
    ([1], [1]),
    ([5, 64, 65, 200], [1, 1, 1, 1]),
    ([130, 4, 67, 0, 3], [4, 4, 4, 4, 4]),             # one idle, one shorter than its tokens
    ([100, 33, 300, 64, 129], [37, 0, 170, 64, 1]),    # ragged, one without new tokens
    ([257, 31], [257, 30]),
    ([70, 20, 12, 7], [12, 12, 12, 12]),               # equal runs over a block's end; one too short
    ([200, 90], [80, 80]),
]


def place_args(lens, new, ragged):
    n = torch.tensor(lens, dtype=torch.int32)
    starts = torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int32)
    wide = torch.stack((n, n * 0 - 9), 1).to(dev())
    return wide[:, 0], starts.to(dev()) if ragged else None


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("D,bs,H,rot,offset,interleaved,name", [
    (128, 64, 8, 64, 0, False, "bf16"),
    (64, 32, 3, 32, 32, True, "f16"),
    (192, 128, 17, 64, 128, False, "bf16"),
    (128, 64, 0, 0, 0, False, "f32"),        # keys alone, no rotation
    (64, 32, 2, 20, 3, False, "f32"),        # single elements
])
def test_index_prepare(case, D, bs, H, rot, offset, interleaved, name):
    clean()
    lens, new = CASES[case]
    g = gen(case * 100 + D)
    T = sum(new)
    rows, blocks = pages_for(lens, bs, g)
    table = idx.rotary_table(512, rot) if rot else None
    dt = DTYPES[name]
    k = (torch.randn(T, D + 8, generator=g) * 3).to(dt).to(dev())[:, :D]
    k[0] = 0.0  # a row of zeros has a scale
    q = torch.randn(T, H + 2, D, generator=g).to(dt).to(dev())[:, 2:] if H else None
    w = (torch.rand(T, H, generator=g) * 2 - 1).to(dev()) if H else None
    pool = torch.randint(256, (blocks, bs * (D + 4)), generator=g, dtype=torch.uint8).to(dev())
    before = pool.clone()
    bt = torch.tensor([r + [10 ** 6] for r in rows], dtype=torch.int32).to(dev())[:, :-1]
    seq, starts = place_args(lens, new, len(set(new)) > 1)
    got = idx.index_prepare(k, pool, bt, seq, token_starts=starts, q=q, weights=w, table=table,
                            interleaved=interleaved, rot_offset=offset)
    clean()
    places = plain.placement(lens, new)
    pos = [p for _, p in places]
    turn = lambda x: plain.rotate(f64(x), pos, f64(table), interleaved, offset) if rot else f64(x)  # noqa: E731
    mine, want = pool.cpu().numpy(), before.cpu().numpy()
    kk = turn(k[:, None])[:, 0]

    def check_row(bytes8, scale, x):
        s = plain.row_scale(x)
        # The scale: a division and (rotated) three roundings of its largest element.
        assert abs(float(scale) - s) <= 2.0 ** -21 * s
        v = plain.E4M3[bytes8] * float(scale)
        # Half a unit of e4m3 (2^-4 of the value, 2^-10 of the scale below its normals).
        lim = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) * (1 + 2.0 ** -18) + 2.0 ** -20 * s
        assert (np.abs(v - x) <= lim).all()

    for t, (b, p) in enumerate(places):
        if p < 0:
            continue
        page, at = rows[b][p // bs], p % bs
        sc = mine[page, bs * D + 4 * at:bs * D + 4 * at + 4]
        check_row(mine[page, at * D:(at + 1) * D], sc.copy().view(np.float32)[0], kk[t])
        want[page, at * D:(at + 1) * D] = mine[page, at * D:(at + 1) * D]
        want[page, bs * D + 4 * at:bs * D + 4 * at + 4] = sc
    assert (mine == want).all(), "a byte outside the new tokens' rows changed"
    if not H:
        assert got is None
        return
    q8, wo = got
    qq = turn(q)
    q8, wo, w = q8.view(torch.uint8).cpu().numpy(), f64(wo), f64(w)
    for t in range(T):
        for h in range(H):
            scale = np.float32(plain.row_scale(qq[t, h]))
            assert abs(wo[t, h] - w[t, h] * scale) <= 2.0 ** -20 * abs(w[t, h] * scale)
            check_row(q8[t, h], scale, qq[t, h])


def test_index_prepare_feeds_the_logits():
    """What index_prepare writes is what logits_fp8 reads: the logits of the prepared inputs
    against the oracle's on the same bytes, and against the unquantised formula within e4m3."""
    lens, bs, D, H = [70, 200, 0], 64, 128, 64
    g = gen(8)
    rows, blocks = pages_for(lens, bs, g)
    bt = torch.tensor(rows, dtype=torch.int32).to(dev())
    seq = torch.tensor(lens, dtype=torch.int32).to(dev())
    pool = torch.zeros(blocks, bs * (D + 4), dtype=torch.uint8, device=dev())
    starts = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32).to(dev())
    k = torch.randn(sum(lens), D, generator=g).bfloat16().to(dev())
    assert idx.index_prepare(k, pool, bt, seq, token_starts=starts) is None
    q = torch.randn(3, H, D, generator=g).bfloat16().to(dev())
    w = (torch.rand(3, H, generator=g) * 2 - 1).to(dev())
    last = torch.stack([k[max(int(s) - 1, 0)] for s in starts[1:]])
    q8, wo = idx.index_prepare(last, pool, bt, seq, q=q, weights=w)  # (writes the last keys again)
    out = idx.logits_fp8(q8.view(3, 1, H, D), pool, wo, bt, seq, 256)
    clean()
    ref, tol = oracle.paged_logits(q8.view(torch.uint8).view(3, 1, H, D).cpu(), pool.cpu(), wo.cpu(), bt.cpu(), seq.cpu(), 256,
                                   block_size=bs)
    for b, n in enumerate(lens):
        if not n:
            continue
        got = f64(out[b, :n])
        assert (np.abs(got - ref[b, :n]) <= 2e-6 * tol[b, :n] + 1e-7).all()
        kk = f64(k[int(starts[b]):int(starts[b + 1])])
        s = np.maximum(f64(q[b]) @ kk.T, 0.0)
        true = f64(w[b]) @ s
        # Each product of two e4m3 roundings is off by at most 2^-4 + 2^-4 + 2^-8 of itself.
        far = np.abs(f64(w[b])) @ (np.abs(f64(q[b])) @ np.abs(kk).T) * 0.13
        assert (np.abs(got - true) <= far).all()


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("D,bs,H,rot,offset,interleaved,name", [
    (128, 64, 8, 64, 0, False, "bf16"),
    (64, 32, 3, 32, 32, True, "f16"),
    (128, 128, 1, 128, 0, False, "f32"),
    (64, 64, 5, 0, 0, False, "bf16"),
    (64, 32, 2, 20, 3, True, "f32"),         # single elements
])
def test_kv_append(case, D, bs, H, rot, offset, interleaved, name):
    clean()
    lens, new = CASES[case]
    g = gen(case * 10 + D + bs)
    T = sum(new)
    rows, blocks = pages_for(lens, bs, g)
    table = idx.rotary_table(512, rot) if rot else None
    dt = DTYPES[name]
    # Strided views; magnitudes from 2^-6 to 2^6, so that some blocks have to grow and some do not.
    mag = torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g).float())
    k = (torch.randn(T, H, D + 8, generator=g) * mag).to(dt).to(dev())[:, :, :D]
    v = (torch.randn(T, H + 1, D, generator=g) * mag).to(dt).to(dev())[:, 1:]
    pools = [torch.randint(256, (blocks, H, bs, D), generator=g, dtype=torch.uint8) for _ in range(2)]
    for p in pools:
        p[p == 255] = 254  # NaN only where it is asked for
        p[p == 127] = 126
    scales = [torch.exp2(torch.randint(-14, 0, (blocks, H), generator=g).float()) for _ in range(2)]
    kp, vp = (p.to(dev()).view(torch.float8_e4m3fn) for p in pools)
    ks, vs = (s.to(dev()) for s in scales)
    seq, starts = place_args(lens, new, len(set(new)) > 1)
    bt = torch.tensor([r + [-5] for r in rows], dtype=torch.int32).to(dev())[:, :-1]
    idx.kv_append(k, v, kp, vp, ks, vs, bt, seq, token_starts=starts, table=table,
                  interleaved=interleaved, rot_offset=offset)
    clean()
    pos = [p for _, p in plain.placement(lens, new)]
    kk = plain.rotate(f64(k), pos, f64(table), interleaved, offset) if rot else f64(k)
    fresh = {(rows[b][p // bs], p % bs): t for t, (b, p) in enumerate(plain.placement(lens, new)) if p >= 0}
    for x, pool, sc, got, got_s, exact in ((kk, pools[0], scales[0], kp, ks, not rot),
                                           (f64(v), pools[1], scales[1], vp, vs, True)):
        ref, ref_s = plain.E4M3[pool.numpy()], sc.double().numpy()
        plain.append(x, ref, ref_s, rows, lens, new, bs)
        mine = values8(got)
        assert (f64(got_s) == ref_s).all()
        if exact:  # no rotation: the same float32 values, the same roundings
            assert (mine == ref).all()
            continue
        for (page, at), t in fresh.items():
            s = ref_s[page][:, None]
            lim = np.maximum(2.0 ** -4 * np.abs(x[t]), 2.0 ** -10 * s) * (1 + 2.0 ** -18) \
                + 2.0 ** -21 * np.abs(x[t]).max(-1, keepdims=True)
            assert (np.abs(mine[page, :, at] * s - x[t]) <= lim).all()
            mine[page, :, at] = ref[page, :, at] = 0.0
        assert (mine == ref).all(), "a token that was there differs"


def test_kv_append_token_by_token_equals_all_at_once():
    """Growing a block's scale is exact for what stays normal: values one decade apart, appended
    one at a time, end as if written together."""
    D, bs, H = 64, 32, 2
    g = gen(4)
    x = torch.randn(40, H, D, generator=g) * torch.logspace(-1, 0, 40)[:, None, None]
    x = torch.where(x.abs() < 0.01, 0.01, x).bfloat16().to(dev())
    bt = torch.tensor([[1, 0]], dtype=torch.int32, device=dev())
    ends = []
    for step in (1, 40):
        kp, vp = (torch.zeros(2, H, bs, D, dtype=torch.float8_e4m3fn, device=dev()) for _ in range(2))
        ks, vs = (torch.ones(2, H, device=dev()) for _ in range(2))
        for t in range(0, 40, step):
            seq = torch.tensor([t + step], dtype=torch.int32, device=dev())
            idx.kv_append(x[t:t + step], x[t:t + step], kp, vp, ks, vs, bt, seq)
        ends.append((values8(kp) * f64(ks)[:, :, None, None], f64(ks)))
    clean()
    assert (ends[0][1] == ends[1][1]).all() and (ends[0][0] == ends[1][0]).all()


def test_writers_skip_and_flag_bad_pages_and_positions():
    D, bs, H = 64, 32, 2
    g = gen(5)
    bt = torch.tensor([[0, 9], [-1, 1]], dtype=torch.int32, device=dev())   # 9 and -1 are no pages
    seq = torch.tensor([40, 40], dtype=torch.int32, device=dev())           # tokens 0 .. 39 of each
    x = torch.randn(80, H, D, generator=g).bfloat16().to(dev())
    kp, vp = (torch.zeros(2, H, bs, D, dtype=torch.uint8, device=dev()) for _ in range(2))
    ks, vs = (torch.zeros(2, H, device=dev()) for _ in range(2))
    table = idx.rotary_table(8, 32)
    clean()
    idx.kv_append(x, x, kp, vp, ks, vs, bt, seq)
    clean(idx.IDX_DEV_BAD_PAGE)
    assert (values8(kp)[0] * f64(ks)[0][:, None, None] != 0).mean() > 0.9
    assert (values8(kp)[1, :, 8:] == 0).all() and (values8(kp)[1, :, :8] != 0).any()
    pool = torch.zeros(2, bs * (D + 4), dtype=torch.uint8, device=dev())
    idx.index_prepare(x[:, 0], pool, bt, seq, table=table)
    clean(idx.IDX_DEV_BAD_PAGE | idx.IDX_DEV_BAD_POSITION)
    idx.kv_append(x, x, kp, vp, ks, vs, bt[:, :1], seq)                     # a table too narrow
    clean(idx.IDX_DEV_BAD_PAGE)
    # Rows past the last request's are padding: nothing is written, nothing flagged.
    kp.zero_()
    starts = torch.tensor([0, 2, 2], dtype=torch.int32, device=dev())
    idx.kv_append(x[:6], x[:6], kp, vp, ks, vs, bt, torch.tensor([2, 0], dtype=torch.int32, device=dev()),
                  token_starts=starts)
    clean()
    assert (kp[0, :, 2:] == 0).all() and (kp[1] == 0).all() and (kp[0, :, :2] != 0).any()


def test_writers_with_what_is_not_finite():
    """Infinities are held at the largest value, NaN as NaN; neither has a say in the scale."""
    D, bs = 64, 32
    x = torch.ones(1, 1, D)
    x[0, 0, 1], x[0, 0, 2], x[0, 0, 3], x[0, 0, 4] = math.inf, -math.inf, math.nan, -3.5
    x = x.to(dev())
    bt = torch.zeros(1, 1, dtype=torch.int32, device=dev())
    seq = torch.ones(1, dtype=torch.int32, device=dev())
    kp, vp = (torch.zeros(1, 1, bs, D, dtype=torch.uint8, device=dev()) for _ in range(2))
    ks, vs = (torch.full((1, 1), math.nan, device=dev()) for _ in range(2))
    idx.kv_append(x, x, kp, vp, ks, vs, bt, seq)
    pool = torch.zeros(1, bs * (D + 4), dtype=torch.uint8, device=dev())
    q8, w = idx.index_prepare(x[:, 0], pool, bt, seq, q=x, weights=torch.ones(1, 1, device=dev()))
    clean()
    for row, s in ((values8(kp)[0, 0, 0], 2.0 ** -7), (values8(q8)[0, 0], 3.5 / 448)):
        assert row[1] == 448 and row[2] == -448 and math.isnan(row[3]) and row[4] == -3.5 / s
        assert row[0] == plain.e4m3(1 / s)
    assert float(ks) == 2.0 ** -7 and float(w) == np.float32(3.5 / 448)


# ---- attention -----------------------------------------------------------------------------------

def attention_case(lens, n, H, Hkv, D, bs, name, seed, poison=True, qmag=1.0):
    """Inputs whose unseen positions, unused pages and scales all hold NaN."""
    g = gen(seed)
    rows, blocks = pages_for(lens, bs, g)
    k, v = (torch.randn(blocks, Hkv, bs, D, generator=g).mul(60).to(torch.float8_e4m3fn)
            .view(torch.uint8) for _ in range(2))
    ks, vs = (torch.rand(blocks, Hkv, generator=g) * 0.03 + 0.005 for _ in range(2))
    if poison:
        used = torch.zeros(blocks, bs, dtype=torch.bool)
        for b, m in enumerate(lens):
            for p in range(m):
                used[rows[b][p // bs], p % bs] = True
        for t in (k, v):
            t.permute(0, 2, 1, 3)[~used] = 0x7F
        for s in (ks, vs):
            s[~used.any(1)] = math.nan
    q = (torch.randn(len(lens), n, H + 1, D + 8, generator=g) * qmag).to(DTYPES[name])
    return dict(q=q.to(dev())[:, :, 1:, :D], k=k.to(dev()).view(torch.float8_e4m3fn),
                v=v.to(dev()).view(torch.float8_e4m3fn), ks=ks.to(dev()), vs=vs.to(dev()),
                bt=torch.tensor([r + [10 ** 6] for r in rows], dtype=torch.int32).to(dev())[:, :-1],
                seq=torch.tensor([[m, -1] for m in lens], dtype=torch.int32).to(dev())[:, 0],
                rows=rows, lens=lens, bs=bs, name=name)


def run_attention(c, **more):
    B, n, H, _ = c["q"].shape
    lse = torch.full((B, n, H), math.nan, device=dev())
    out = idx.attention_fp8(c["q"], c["k"], c["v"], c["ks"], c["vs"], c["bt"], c["seq"], lse=lse, **more)
    torch.cuda.synchronize()
    return out, lse


def check_attention(c, out, lse, picked=None, scale=None):
    """Tolerance.  A query element is held to 2^-18 of its row's largest magnitude (bfloat16 is
    then exact above that; float16 to 2^-19 with one part more), products are exact, sums are
    float32: the scores are off by dz at most.  A weight is held to 2^-8 of itself (float16 2^-12)
    or 2^-17 of the largest, so the weighted sum is off by (2 dz + that) * sum w |v| plus
    2^-17 * sum |v| / sum_p exp(z_p - max).  The output is rounded once."""
    name, D = c["name"], c["q"].shape[3]
    scale = D ** -0.5 if scale is None else scale
    q, k, v, ks, vs = f64(c["q"]), values8(c["k"]), values8(c["v"]), f64(c["ks"]), f64(c["vs"])
    ref, ref_lse, mag, seen = plain.attention(q, k, v, ks, vs, c["rows"], c["lens"], c["bs"], scale, picked)
    B, n, H, _ = q.shape
    G = H // k.shape[1]
    got, got_lse = f64(out), f64(lse)
    w_rel = 2.0 ** -8 if name == "bf16" else 2.0 ** -12
    for b in range(B):
        for t in range(n):
            pos = np.array(seen[b * n + t], dtype=int)
            if not pos.size:
                assert (got[b, t] == 0).all() and (got_lse[b, t] == -np.inf).all()
                continue
            page = np.asarray(c["rows"][b])[pos // c["bs"]]
            for h in range(H):
                kk = np.abs(k[page, h // G, pos % c["bs"]] * ks[page, h // G][:, None])
                vv = np.abs(v[page, h // G, pos % c["bs"]] * vs[page, h // G][:, None])
                dz = abs(scale) * np.max(2.0 ** -18 * np.abs(q[b, t, h]).max() * kk.sum(1)
                                    + 2.0 ** -17 * (kk @ np.abs(q[b, t, h])))
                top = math.exp(-ref_lse[b, t, h] + np.max(scale * ((k[page, h // G, pos % c["bs"]] * ks[page, h // G][:, None]) @ q[b, t, h])))
                lim = (2 * dz + w_rel + 2.0 ** -18) * mag[b, t, h] + 2.0 ** -17 * top * vv.sum(0)
                lim = lim + HALF_ULP[name] * (np.abs(ref[b, t, h]) + lim) + FLOOR[name]
                err = np.abs(got[b, t, h] - ref[b, t, h])
                assert (err <= lim).all(), (b, t, h, float(np.max(err / lim)))
                assert abs(got_lse[b, t, h] - ref_lse[b, t, h]) <= dz + 2.0 ** -20 * (1 + abs(ref_lse[b, t, h])) + 2.0 ** -18


SHAPES = [  # H, Hkv, D, block, dtype
    (8, 8, 128, 64, "bf16"),     # a head of its own for each query head
    (16, 2, 128, 64, "bf16"),
    (6, 2, 64, 32, "f16"),       # groups of three
    (64, 1, 128, 128, "f16"),
    (70, 2, 64, 64, "bf16"),     # groups of 35
    (13, 1, 128, 32, "f16"),
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


@pytest.mark.parametrize("num_sms", [1, 3, 40])
def test_attention_split_any_way(num_sms):
    """Few CTAs walk many requests each; many CTAs share one request."""
    for lens in (LENS, [1500], [5] * 70):
        c = attention_case(lens, 2, 16, 2, 128, 64, "bf16", 17)
        out, lse = run_attention(c, num_sms=num_sms)
        check_attention(c, out, lse)
    clean()


def test_attention_among_idle_slots():
    """A fixed batch most of whose slots are idle, in stretches longer than a warp."""
    lens = [0] * 70 + [40] + [0] * 33 + [300, 0, 5] + [0] * 100 + [129] + [0] * 40
    c = attention_case(lens, 1, 8, 2, 64, 32, "bf16", 47)
    for num_sms in (1, 0):
        out, lse = run_attention(c, num_sms=num_sms)
        check_attention(c, out, lse)
    cand, ranges, picked = selections(c, 30, gen(3))
    out, lse = run_attention(c, candidates=cand, ranges=ranges)
    check_attention(c, out, lse, picked)
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


def test_attention_ranges_outside_the_slots():
    """A range is held to the slots there are; an empty or reversed one gives a row of zeros."""
    c = attention_case([200, 200, 200], 1, 8, 1, 64, 32, "bf16", 5)
    cand, _, _ = selections(c, 16, gen(1))
    cand[:, :, 0] = torch.arange(40, device=dev(), dtype=torch.int32)
    ranges = torch.tensor([[-7, 30, 12], [5, 99, 12]], dtype=torch.int32, device=dev())
    out, lse = run_attention(c, candidates=cand, ranges=ranges)
    check_attention(c, out, lse, [list(range(5)), list(range(30, 40)), []])
    clean()


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_attention_with_large_scores(name):
    """Scores of a few hundred: one position carries a row, and others' weights vanish."""
    c = attention_case([5, 700, 130], 1, 16, 2, 128, 64, name, 23, qmag=30.0)
    out, lse = run_attention(c)
    check_attention(c, out, lse)
    out, lse = run_attention(c, softmax_scale=0.0)
    check_attention(c, out, lse, scale=0.0)
    out, lse = run_attention(c, softmax_scale=-0.05)
    check_attention(c, out, lse, scale=-0.05)
    clean()


def test_attention_with_block_scales_far_apart():
    """Blocks whose scales differ by 2^24 in one tile; a block with scale 0; zero queries."""
    c = attention_case([256, 300], 1, 8, 1, 128, 32, "bf16", 29)
    for b in range(2):
        for j, page in enumerate(c["rows"][b][:8]):
            c["vs"][page] = 2.0 ** (-12 * (j % 3))
            c["ks"][page] = 0.0 if j == 2 else 0.01 * 2.0 ** (-8 * (j % 2))
    c["q"][1, 0, 3] = 0.0
    out, lse = run_attention(c)
    check_attention(c, out, lse)
    clean()


@pytest.mark.parametrize("H,Hkv,D,bs,name", [(8, 1, 128, 64, "bf16"), (64, 2, 64, 32, "f16")])
def test_attention_with_negative_and_zero_scales(H, Hkv, D, bs, name):
    """Scales of either sign; a block whose values all count as 0; all of them 0."""
    c = attention_case([300, 64, 129], 1, H, Hkv, D, bs, name, 53)
    flip = (torch.arange(c["vs"].numel(), device=dev()) % 3 == 0).view_as(c["vs"])
    c["vs"] = torch.where(flip, -c["vs"], c["vs"])
    c["ks"] = torch.where(flip.roll(1, 0), -c["ks"], c["ks"])
    c["vs"][c["rows"][0][1]] = 0.0
    out, lse = run_attention(c)
    check_attention(c, out, lse)
    for page in c["rows"][2][:-(-129 // bs)]:
        c["vs"][page] = 0.0
    out, lse = run_attention(c)
    check_attention(c, out, lse)
    assert (out[2] == 0).all()
    clean()


def test_attention_never_sees_what_a_draft_slot_does_not():
    """NaN in the values and keys of the newest tokens reaches the slots that see them, and only
    those."""
    n, lens = 4, [130, 64, 6]
    c = attention_case(lens, n, 8, 2, 128, 64, "bf16", 31)
    base, _ = run_attention(c)
    for b, m in enumerate(lens):
        p = m - 2  # seen by slots 2 and 3
        c["v"].view(torch.uint8)[c["rows"][b][p // 64], 0, p % 64, 5] = 0x7F
        c["k"].view(torch.uint8)[c["rows"][b][p // 64], 1, p % 64, 7] = 0xFF
    out, _ = run_attention(c)
    clean()
    assert torch.equal(out[:, :2], base[:, :2])
    assert torch.isnan(out[:, 2:, :4, 5]).all() and torch.isnan(out[:, 2:, 4:]).all()
    keep = [d for d in range(128) if d != 5]
    assert torch.equal(out[:, 2:, :4][..., keep], base[:, 2:, :4][..., keep])


def test_attention_flags_bad_pages():
    """A block id outside the pool and a table too narrow: those positions are passed over."""
    c = attention_case([200, 130], 1, 8, 2, 64, 32, "bf16", 37)
    c["bt"][0, 2] = 10 ** 6
    c["bt"][1, 0] = -1
    out, lse = run_attention(c)
    clean(idx.IDX_DEV_BAD_PAGE)
    picked = [[p for p in range(200) if p // 32 != 2], list(range(32, 130))]
    check_attention(c, out, lse, picked)
    c["bt"] = torch.tensor(c["rows"], dtype=torch.int32).to(dev())[:, :3]
    out, lse = run_attention(c)
    clean(idx.IDX_DEV_BAD_PAGE)
    check_attention(c, out, lse, [list(range(96)), list(range(96))])
    cand, ranges, picked = selections(c, 50, gen(2))
    out, lse = run_attention(c, candidates=cand, ranges=ranges)
    clean(idx.IDX_DEV_BAD_PAGE)
    check_attention(c, out, lse, [[p for p in row if p < 96] for row in picked])


def test_attention_past_32_bits():
    """Pages past 2^31 bytes of a pool, and of the slots' offsets."""
    D, bs, Hkv = 128, 64, 1
    blocks = (1 << 31) // (bs * D) + 64
    c = attention_case([150, 90], 1, 4, Hkv, D, bs, "bf16", 41)
    big = {}
    for name in ("k", "v"):
        pool = torch.empty(blocks, Hkv, bs, D, dtype=torch.uint8, device=dev())
        pool[-c["k"].shape[0]:] = c[name].view(torch.uint8)
        big[name] = pool.view(torch.float8_e4m3fn)
    first = blocks - c["k"].shape[0]
    wide = {}
    for name in ("ks", "vs"):
        wide[name] = torch.full((blocks, Hkv), math.nan, device=dev())
        wide[name][first:] = c[name]
    out, lse = run_attention({**c, **big, **wide, "bt": torch.tensor(c["rows"], dtype=torch.int32).to(dev()) + first})
    clean()
    check_attention(c, out, lse)
    # The writers at the same pages: read back through the attention's own indexing.
    x = torch.randn(240, Hkv, D, generator=gen(1)).bfloat16().to(dev())
    starts = torch.tensor([0, 150, 240], dtype=torch.int32, device=dev())
    bt = torch.tensor(c["rows"], dtype=torch.int32).to(dev())
    small = [torch.zeros_like(c["k"]) for _ in range(2)], [torch.zeros_like(c["ks"]) for _ in range(2)]
    idx.kv_append(x, x, *small[0], *small[1], bt, c["seq"], token_starts=starts)
    idx.kv_append(x, x, big["k"], big["v"], wide["ks"], wide["vs"], bt + first, c["seq"], token_starts=starts)
    clean()
    used = sorted({p for b, m in enumerate(c["lens"]) for p in c["rows"][b][:-(-m // bs)]})
    for p in used:
        m = max(c["lens"][b] - bs * r.index(p) for b, r in enumerate(c["rows"]) if p in r[:-(-c["lens"][b] // bs)])
        for a, b in zip(small[0], (big["k"], big["v"])):
            assert torch.equal(a[p, :, :m].view(torch.uint8), b[first + p, :, :m].view(torch.uint8))


def test_attention_on_another_stream_and_in_a_graph():
    c = attention_case(LENS, 2, 16, 2, 128, 64, "bf16", 43)
    want, _ = run_attention(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = idx.attention_fp8(c["q"], c["k"], c["v"], c["ks"], c["vs"], c["bt"], c["seq"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    seq = c["seq"].clone()
    with torch.cuda.graph(graph):
        held = idx.attention_fp8(c["q"], c["k"], c["v"], c["ks"], c["vs"], c["bt"], seq)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, want)
    seq.copy_(torch.tensor([max(0, m - 7) for m in LENS], dtype=torch.int32))  # lengths of a later replay
    graph.replay()
    short = dict(c, seq=seq, lens=[max(0, m - 7) for m in LENS])
    want, _ = run_attention(short)
    assert torch.equal(held, want)
    clean()


def test_append_then_attend():
    """Tokens written by kv_append and read by attention_fp8, against the attention over the
    unquantised keys and values: off by no more than e4m3 holds."""
    lens, D, bs, H, Hkv = [90, 200], 64, 32, 8, 2
    g = gen(9)
    rows, blocks = pages_for(lens, bs, g)
    table = idx.rotary_table(256, 32)
    T = sum(lens)
    k, v = (torch.randn(T, Hkv, D, generator=g).bfloat16().to(dev()) for _ in range(2))
    kp, vp = (torch.full((blocks, Hkv, bs, D), 0x7F, dtype=torch.uint8, device=dev()) for _ in range(2))
    ks, vs = (torch.full((blocks, Hkv), math.nan, device=dev()) for _ in range(2))
    bt = torch.tensor(rows, dtype=torch.int32).to(dev())
    seq = torch.tensor(lens, dtype=torch.int32).to(dev())
    starts = torch.tensor([0, 90, 290], dtype=torch.int32).to(dev())
    idx.kv_append(k, v, kp, vp, ks, vs, bt, seq, token_starts=starts, table=table, rot_offset=32)
    q = torch.randn(2, 1, H, D, generator=g).bfloat16().to(dev())
    out = f64(idx.attention_fp8(q, kp, vp, ks, vs, bt, seq))
    clean()
    kk = plain.rotate(f64(k), [p for _, p in plain.placement(lens, lens)], f64(table), False, 32)
    for b in range(2):
        a, e = int(starts[b]), int(starts[b + 1])
        for h in range(H):
            z = kk[a:e, h // 4] @ f64(q)[b, 0, h] / 8.0
            w = np.exp(z - z.max())
            w /= w.sum()
            ref = w @ f64(v)[a:e, h // 4]
            # e4m3 puts an error of 2^-5 rms at most on each of 64 products (|z| off by 0.05 rms)
            # and on each value; ten times that, over the weights' spread.
            lim = 10 * 0.09 * np.sqrt((w ** 2) @ f64(v)[a:e, h // 4] ** 2) + 0.01
            assert (np.abs(out[b, 0, h] - ref) <= lim).all()


def test_kv_append_long_runs_equal_their_parts():
    """A prompt long enough that a CTA takes several heads, in one call and in calls of a few blocks
    each: the same bytes and scales."""
    T, H, D, bs = 21000, 8, 64, 64
    g = gen(12)
    blocks = -(-T // bs)
    x = (torch.randn(T, H, D, generator=g) * torch.exp2(torch.randint(-4, 5, (T, 1, 1), generator=g).float())).bfloat16().to(dev())
    y = torch.randn(T, H, D, generator=g).bfloat16().to(dev())
    table = idx.rotary_table(T, 32)
    bt = torch.randperm(blocks, generator=g).int()[None].to(dev())
    ends = []
    for step in (T, 40 * bs):
        kp, vp = (torch.zeros(blocks, H, bs, D, dtype=torch.uint8, device=dev()) for _ in range(2))
        ks, vs = (torch.zeros(blocks, H, device=dev()) for _ in range(2))
        for a in range(0, T, step):
            e = min(a + step, T)
            idx.kv_append(x[a:e], y[a:e], kp, vp, ks, vs, bt, torch.tensor([e], dtype=torch.int32, device=dev()),
                          token_starts=torch.tensor([0, e - a], dtype=torch.int32, device=dev()), table=table)
        ends.append((kp, vp, ks, vs))
    clean()
    for a, b in zip(*ends):
        assert torch.equal(a, b)
    v = values8(ends[0][1]) * f64(ends[0][3])[:, :, None, None]
    order = bt[0].cpu().numpy()
    whole = v[order].transpose(0, 2, 1, 3).reshape(-1, H, D)[:T]
    s = f64(ends[0][3])[order].repeat(bs, 0)[:T, :, None]
    assert (np.abs(whole - f64(y)) <= np.maximum(2.0 ** -4 * np.abs(f64(y)), 2.0 ** -10 * s)).all()


@pytest.mark.parametrize("which", ["tables", "lens"])
def test_expanded_tables_and_lengths_are_refused(which):
    B, H, D, bs = 3, 2, 64, 32
    pool = torch.zeros(8, H, bs, D, dtype=torch.uint8, device="cuda")
    sc = torch.ones(8, H, device="cuda")
    bt = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
    sl = torch.ones(B, dtype=torch.int32, device="cuda")
    if which == "tables":
        bt = bt[:1].expand(B, 2)
    else:
        sl = sl[:1].expand(B)
    x = torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda")
    fused = torch.zeros(8, bs * (D + 4), dtype=torch.uint8, device="cuda")
    for call in (lambda: idx.attention_fp8(x[:, None], pool, pool, sc, sc, bt, sl),
                 lambda: idx.kv_append(x, x, pool, pool, sc, sc, bt, sl),
                 lambda: idx.index_prepare(x[:, 0], fused, bt, sl)):
        with pytest.raises(ValueError, match="expanded"):
            call()
    # One request: the strides of its only row mean nothing.
    idx.attention_fp8(x[:1, None], pool, pool, sc, sc, bt[:1], sl[:1].expand(1))

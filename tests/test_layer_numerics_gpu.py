"""The operators around the indexer where their arithmetic is narrow: e4m3 codes of quotients, weights
far below a row's largest, what is not finite, offsets past 32 bits.  Against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import layer_plain as plain
import paged_fp8_mqa_gb300 as idx

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev():
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.detach().cpu().double().numpy()


def values8(t):
    return plain.E4M3[t.detach().view(torch.uint8).cpu().numpy()]


def clean(bits=0):
    torch.cuda.synchronize()
    assert idx.device_status(clear=True) == bits


# ---- index rows ----------------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rot", [0, 64])
def test_index_rows_hold_the_quotients(name, rot):
    """A code is the e4m3 nearest to the float32 quotient of the (turned) element by the scale that is
    stored beside it: no code may be its neighbour's."""
    clean()
    B, H, D, bs = 1024, 16, 128, 64
    g = gen(61)
    k = torch.randn(B, D, generator=g).to(DTYPES[name]).to(dev())
    q = (torch.randn(B, H, D, generator=g) * torch.exp2(torch.randint(-3, 4, (B, H, 1), generator=g).float())) \
        .to(DTYPES[name]).to(dev())
    pool = torch.zeros(B, bs * (D + 4), dtype=torch.uint8, device=dev())
    bt = torch.arange(B, dtype=torch.int32, device=dev())[:, None]
    seq = torch.arange(B, dtype=torch.int32, device=dev()) % bs + 1
    table = idx.rotary_table(bs, rot) if rot else None
    q8, scale = idx.index_prepare(k, pool, bt, seq, q=q, weights=torch.ones(B, H, device=dev()), table=table)
    clean()
    at = (seq.cpu().numpy() - 1)
    cs = table.cpu().numpy()[at] if rot else None

    def turned(x):  # float32 [B, ..., D], each product rounded before the sum
        x = x.float().cpu().numpy()
        if not rot:
            return x
        y, h = x.copy(), rot // 2
        c, s = (cs[..., i].reshape(B, *([1] * (x.ndim - 2)), h) for i in (0, 1))
        y[..., :h] = x[..., :h] * c - x[..., h:rot] * s
        y[..., h:rot] = x[..., h:rot] * c + x[..., :h] * s
        return y

    pool = pool.cpu().numpy()
    k8 = np.stack([pool[b, a * D:(a + 1) * D] for b, a in enumerate(at)])
    ks = np.stack([pool[b, bs * D + 4 * a:bs * D + 4 * a + 4] for b, a in enumerate(at)]).view(np.float32)[:, 0]
    for codes, x, s in ((q8.view(torch.uint8).cpu().numpy(), turned(q), scale.cpu().numpy()), (k8, turned(k), ks)):
        want = plain.e4m3(x / s[..., None])
        assert x.dtype == np.float32 and s.dtype == np.float32
        assert (plain.E4M3[codes] == want).all(), int((plain.E4M3[codes] != want).sum())


def test_index_rows_with_an_infinity_hold_the_quotients():
    D, bs = 64, 32
    x = torch.randn(64, D, generator=gen(3)) * 3
    x[:, 5], x[:, 9], x[:, 11] = math.inf, -math.inf, math.nan
    x = x.to(dev())
    pool = torch.zeros(64, bs * (D + 4), dtype=torch.uint8, device=dev())
    bt = torch.arange(64, dtype=torch.int32, device=dev())[:, None]
    seq = torch.ones(64, dtype=torch.int32, device=dev())
    idx.index_prepare(x, pool, bt, seq)
    clean()
    pool = pool.cpu().numpy()
    scale = pool[:, bs * D:bs * D + 4].copy().view(np.float32)
    want = plain.e4m3(x.cpu().numpy() / scale)
    np.testing.assert_array_equal(plain.E4M3[pool[:, :D]], want)


def test_index_rows_keep_the_signs_of_zeros():
    D, bs = 64, 32
    x = torch.zeros(2, D)
    x[:, ::3], x[1, 5], x[1, 7] = -0.0, -2.0, -1e-30
    pool = torch.zeros(2, bs * (D + 4), dtype=torch.uint8, device=dev())
    seq = torch.ones(2, dtype=torch.int32, device=dev())
    bt = torch.arange(2, dtype=torch.int32, device=dev())[:, None]
    q8, _ = idx.index_prepare(x.to(dev()), pool, bt, seq, q=x[:, None].to(dev()), weights=torch.ones(2, 1, device=dev()))
    clean()
    want = torch.signbit(x).numpy()
    assert ((pool.cpu().numpy()[:, :D] >= 0x80) == want).all()
    assert ((q8.view(torch.uint8).cpu().numpy()[:, 0] >= 0x80) == want).all()


def test_index_prepare_writes_the_keys_of_queries_without_heads():
    B, D, bs = 3, 64, 32
    k = torch.randn(B, D, generator=gen(7)).bfloat16().to(dev())
    bt = torch.arange(B, dtype=torch.int32, device=dev())[:, None]
    seq = torch.tensor([1, 9, 32], dtype=torch.int32, device=dev())
    want, got = (torch.zeros(B, bs * (D + 4), dtype=torch.uint8, device=dev()) for _ in range(2))
    idx.index_prepare(k, want, bt, seq)
    q8, w = idx.index_prepare(k, got, bt, seq, q=torch.zeros(B, 0, D, dtype=torch.bfloat16, device=dev()),
                              weights=torch.zeros(B, 0, device=dev()))
    clean()
    assert q8.shape == (B, 0, D) and w.shape == (B, 0)
    assert (want != 0).any() and torch.equal(got, want)


# ---- rotary positions outside the table --------------------------------------------------------------

@pytest.mark.parametrize("name", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,offset", [(64, 32, 16), (30, 10, 3)])   # wide pieces, single elements
@pytest.mark.parametrize("layout", ["plain", "in place"])
def test_rotary_leaves_rows_past_the_table_to_the_bit(name, interleaved, D, rot, offset, layout):
    clean()
    x = torch.randn(3, 3, D, generator=gen(5))
    x[:, :, 1::5], x[:, :, 2::7], x[:, :, 3::11], x[:, :, 4::9] = math.inf, -0.0, math.nan, -math.inf
    x = x.to(DTYPES[name]).to(dev())
    bits = torch.int32 if name == "f32" else torch.int16
    keep = x.clone()
    y = idx.rotary(x, torch.tensor([-1, 10, 2 ** 31 - 1], dtype=torch.int32, device=dev()), idx.rotary_table(10, rot),
                   interleaved=interleaved, rot_offset=offset, out=x if layout == "in place" else None)
    clean(idx.IDX_DEV_BAD_POSITION)
    assert torch.equal(y.view(bits), keep.view(bits))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_is_recorded_by_autograd(interleaved, inverse):
    """The gradient autograd finds is the formula's; a second backward turns again."""
    table = idx.rotary_table(50, 16, scaling="yarn", factor=4.0, original_positions=64)
    pos = torch.tensor([0, 49, 20, 60], dtype=torch.int32, device=dev())   # 60: past the table, left alone
    w = torch.randn(4, 2, 24, generator=gen(2)).to(dev())
    wide = torch.randn(4, 3, 32, generator=gen(1)).to(dev()).requires_grad_()
    x = wide[:, 1:, :24]
    y = idx.rotary(x, pos, table, interleaved=interleaved, rot_offset=8, inverse=inverse)
    assert y.requires_grad
    plain_y = idx.rotary(x.detach(), pos, table, interleaved=interleaved, rot_offset=8, inverse=inverse)
    assert not plain_y.requires_grad and torch.equal(y, plain_y)
    with torch.no_grad():
        assert not idx.rotary(x, pos, table, interleaved=interleaved, rot_offset=8).requires_grad
    up = w.clone().requires_grad_()
    (grad,) = torch.autograd.grad(y, wide, up, create_graph=True)
    turn = f64(table) * ([1, 1] if inverse else [1, -1])
    want = np.zeros((4, 3, 32))
    want[:, 1:, :24] = plain.rotate(f64(w), pos.tolist(), turn, interleaved, 8)
    # Two products and a sum in float32, of a magnitude of at most 1.14 times sqrt(2) max |w|.
    assert np.abs(f64(grad) - want).max() <= 3 * 2.0 ** -24 * 1.14 * 2 * f64(w.abs().max())
    (back,) = torch.autograd.grad(grad, up, wide.detach())
    assert torch.equal(back, plain_y)
    (ones,) = torch.autograd.grad(idx.rotary(x, pos, table, interleaved=interleaved, rot_offset=8).sum(), wide)
    flat = idx.rotary(torch.ones_like(w), pos, table, interleaved=interleaved, rot_offset=8, inverse=True)
    assert torch.equal(ones[:, 1:, :24], flat)
    idx.device_status(clear=True)


# ---- weights far below a row's largest -------------------------------------------------------------

def tail_case(N, H, Hkv, D, bs, name, *, share=None, gap=None, spread, ratio=1.0, n=1, seed=0):
    """Requests of N and of a few positions fewer, whose first position takes `share` of each row's
    weight (or stands `gap` above the mean score of the others) and has the value 0; the
    other values have a mean of 1.  ratio: the first block's value scale over the others' (its values
    are all 0 then)."""
    g = gen(seed)
    lens = [N, N - min(7, N - n - 1)]
    pages = -(-N // bs)
    rows = [torch.randperm(2 * pages, generator=g)]
    rows = torch.stack((rows[0][:pages], rows[0][pages:]))
    k = torch.randn(2 * pages, Hkv, bs, D, generator=g).mul(60).to(torch.float8_e4m3fn)
    v = (torch.randn(2 * pages, Hkv, bs, D, generator=g) + 1).mul(60).to(torch.float8_e4m3fn)
    ks, vs = (torch.full((2 * pages, Hkv), 1.0 / 60) for _ in range(2))
    # Four channels are the first position's alone: its key there and the queries' give it its score.
    k.view(torch.uint8)[..., :4] = 0
    q = torch.randn(2, n, H, D, generator=g) * spread
    q[..., :4] = 16.0
    q = q.to(DTYPES[name])
    aim = gap if gap is not None else math.log(share / (1 - share)) + math.log(N) + spread ** 2 / 2
    code = torch.tensor(aim * D ** 0.5 / 64.0 * 60).to(torch.float8_e4m3fn)
    assert float(code) < 448
    for b in range(2):
        first = rows[b, 0]
        k[first, :, 0] = torch.zeros(Hkv, D).to(torch.float8_e4m3fn)
        k[first, :, 0, :4] = code
        v.view(torch.uint8)[first, :, :bs if ratio != 1 else 1] = 0
        vs[first] *= ratio
    on = lambda t: t.to(dev())  # noqa: E731
    return dict(q=on(q), k=on(k), v=on(v), ks=on(ks), vs=on(vs), bt=on(rows.int()),
                seq=on(torch.tensor(lens, dtype=torch.int32)), rows=rows.numpy(), lens=lens, bs=bs, name=name)


def check_tail(c, picked=False, num_sms=0):
    """The limit is relative to sum w |v|, with no term that grows with the length: a weight is within
    2^-10 of itself (bfloat16; float16 2^-14) or 2^-35 of the row's largest, which 2^-14 covers here; the
    scores are off by dz (a query element to 2^-18 of its row's largest, float32 sums); the output is
    rounded once (a float16 below its normals to 2^-25)."""
    q = c["q"]
    B, n, H, D = q.shape
    more = {}
    if picked:  # everything, in an order of its own
        most = max(c["lens"])
        cand = torch.zeros(B * n, most + 3, 2, dtype=torch.int32)
        ranges = torch.tensor([[1] * (B * n), [1 + c["lens"][r // n] for r in range(B * n)]], dtype=torch.int32)
        for r in range(B * n):
            m = c["lens"][r // n]
            cand[r, 1:1 + m, 0] = torch.randperm(m, generator=gen(r)).int()
        more = dict(candidates=cand.to(dev()), ranges=ranges.to(dev()))
    lse = torch.empty(B, n, H, device=dev())
    out = idx.attention_fp8(q, c["k"], c["v"], c["ks"], c["vs"], c["bt"], c["seq"], lse=lse, num_sms=num_sms, **more)
    clean()
    qq, kk, vv, ks, vs = f64(q), values8(c["k"]), values8(c["v"]), f64(c["ks"]), f64(c["vs"])
    ref, ref_lse, mag, _ = plain.attention(qq, kk, vv, ks, vs, c["rows"], c["lens"], c["bs"], D ** -0.5)
    # |k| is at most 5 sigma of the products' sums here: of N(0, 1) elements, D of them.
    dz = D ** -0.5 * (2.0 ** -18 * np.abs(qq).max(-1) * 1.2 * D + 2.0 ** -17 * np.abs(qq).sum(-1) * 3)
    w_rel, half, floor = (2.0 ** -10, 2.0 ** -8, 0.0) if c["name"] == "bf16" else (2.0 ** -14, 2.0 ** -11, 2.0 ** -25)
    lim = (2 * dz[..., None] + w_rel + 2.0 ** -14) * mag
    lim = lim + half * (np.abs(ref) + lim) + floor
    err = np.abs(f64(out) - ref)
    assert (err <= lim).all(), float((err / np.maximum(mag, 1e-30)).max())
    assert (np.abs(f64(lse) - ref_lse) <= dz + 2.0 ** -17 * (1 + np.abs(ref_lse))).all()


TAIL_SHAPES = [  # H, Hkv, D, block, dtype: every width of rows
    (8, 1, 128, 64, "bf16"), (16, 1, 64, 32, "bf16"), (24, 1, 128, 64, "bf16"), (32, 1, 64, 32, "bf16"),
    (40, 1, 64, 128, "bf16"), (64, 1, 128, 64, "bf16"),
    (8, 1, 64, 32, "f16"), (32, 1, 128, 64, "f16"), (30, 1, 64, 64, "f16"), (64, 1, 128, 64, "f16"),
]


@pytest.mark.parametrize("H,Hkv,D,bs,name", TAIL_SHAPES)
@pytest.mark.parametrize("N,how", [
    (8192, dict(share=0.8, spread=2.0)), (32768, dict(share=0.5, spread=1.0)), (32768, dict(gap=10.0, spread=0.3, ratio=64.0)),
    (32768, dict(gap=8.0, spread=0.3, ratio=256.0)), (4096, dict(gap=13.0, spread=0.5, ratio=256.0)),
    (20, dict(gap=10.0, spread=0.5)), (20, dict(gap=16.0, spread=0.5)), (5, dict(gap=12.0, spread=0.5))])
def test_attention_keeps_small_weights(H, Hkv, D, bs, name, N, how):
    check_tail(tail_case(N, H, Hkv, D, bs, name, **how))


@pytest.mark.parametrize("H,Hkv,D,bs,name", [(8, 1, 128, 64, "bf16"), (32, 1, 64, 32, "bf16"), (16, 1, 128, 64, "f16")])
@pytest.mark.parametrize("share,spread", [(0.5, 0.5), (0.8, 0.5), (0.8, 0.01)])
@pytest.mark.parametrize("num_sms", [1, 0])
def test_attention_keeps_small_weights_over_131072_positions(H, Hkv, D, bs, name, share, spread, num_sms):
    """Two runs for two requests, each uncut, and runs of a few tiles."""
    check_tail(tail_case(131072, H, Hkv, D, bs, name, share=share, spread=spread), num_sms=num_sms)


@pytest.mark.parametrize("H,Hkv,D,bs,name", [(8, 1, 128, 64, "bf16"), (32, 1, 64, 32, "bf16"), (64, 1, 128, 64, "f16")])
@pytest.mark.parametrize("num_sms", [1, 0])
def test_attention_keeps_small_weights_of_a_selection(H, Hkv, D, bs, name, num_sms):
    for N, how in ((8192, dict(share=0.8, spread=1.0)), (2048, dict(gap=10.0, spread=0.3, ratio=64.0)),
                   (2048, dict(gap=14.0, spread=0.3))):
        check_tail(tail_case(N, H, Hkv, D, bs, name, **how), picked=True, num_sms=num_sms)


@pytest.mark.parametrize("n", [2, 4])
def test_attention_keeps_small_weights_of_draft_slots(n):
    check_tail(tail_case(16384, 8, 1, 64, 32, "bf16", share=0.8, spread=0.5, n=n))
    check_tail(tail_case(2048, 16, 2, 128, 64, "bf16", gap=13.0, spread=0.5, n=n))


@pytest.mark.parametrize("H,Hkv,D,bs,name", TAIL_SHAPES)
def test_attention_with_an_outlier_in_the_queries(H, Hkv, D, bs, name):
    """One element of each query 2^19 times the others and no key has its channel: the scores are the
    others' alone.  Elements are exact, or within 2^-31 of the outlier; sums are float32."""
    lens = [300, 77]
    g = gen(H + D)
    blocks = 16
    bt = torch.randperm(blocks, generator=g).int()[:2 * -(-300 // bs)].view(2, -1) if bs > 32 else \
        torch.randperm(20, generator=g).int().view(2, 10)
    blocks = max(blocks, 20)
    k, v = (torch.randn(blocks, Hkv, bs, D, generator=g).mul(60).to(torch.float8_e4m3fn) for _ in range(2))
    k.view(torch.uint8)[..., D // 3] = 0
    ks, vs = (torch.full((blocks, Hkv), 1.0 / 60) for _ in range(2))
    q = torch.randn(2, 1, H, D, generator=g) * 2.0 ** -7
    q[..., D // 3] = 2.0 ** 12
    q = q.to(DTYPES[name])
    scale = 2.0 ** 7 * D ** -0.5
    out = idx.attention_fp8(q.to(dev()), *(t.to(dev()) for t in (k, v, ks, vs, bt)),
                            torch.tensor(lens, dtype=torch.int32, device=dev()), softmax_scale=scale)
    clean()
    kk = values8(k)
    ref, _, mag, _ = plain.attention(f64(q), kk, values8(v), f64(ks), f64(vs), bt.numpy(), lens, bs, scale)
    rest = f64(q)
    rest[..., D // 3] = 0
    sums = np.abs(kk).sum(-1).max() / 60
    dz = scale * (2.0 ** -31 * 2.0 ** 12 * sums + 2.0 ** -17 * np.abs(rest).max() * sums)
    w_rel, half = (2.0 ** -10, 2.0 ** -8) if name == "bf16" else (2.0 ** -14, 2.0 ** -11)
    lim = (2 * dz + w_rel + 2.0 ** -14) * mag
    lim = lim + half * (np.abs(ref) + lim)
    err = np.abs(f64(out) - ref)
    assert (err <= lim).all(), (dz, float((err / mag).max()))


# ---- scales that are not finite --------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,D,bs,name,n", [(8, 2, 128, 32, "bf16", 4), (64, 2, 64, 32, "f16", 1),
                                               (48, 2, 64, 32, "bf16", 3)])
@pytest.mark.parametrize("which,value", [("ks", math.nan), ("vs", math.nan), ("vs", math.inf), ("vs", -math.inf)])
@pytest.mark.parametrize("picked", [False, True])
def test_attention_over_a_scale_that_is_not_finite(H, Hkv, D, bs, name, n, which, value, picked):
    """The rows that see the block are NaN in every element; the others keep their bits."""
    lens = [65 + (n - 1) // 2, 200, 31]
    g = gen(71)
    bt = torch.randperm(16, generator=g).int()[:12].view(3, 4)
    bt = torch.cat((bt, torch.arange(16, 28).int().view(3, 4)), 1)
    k, v = (torch.randn(28, Hkv, bs, D, generator=g).mul(60).to(torch.float8_e4m3fn).to(dev()) for _ in range(2))
    s = {x: (torch.rand(28, Hkv, generator=g) * 0.02 + 0.01).to(dev()) for x in ("ks", "vs")}
    q = torch.randn(3, n, H, D, generator=g).to(DTYPES[name]).to(dev())
    more = {}
    if picked:
        cand = torch.stack([torch.randperm(200, generator=g) for _ in range(3 * n)]).int()
        cand = torch.stack((cand, cand), -1).contiguous().to(dev())
        more = dict(candidates=cand, ranges=torch.tensor([[0] * 3 * n, [200] * 3 * n], dtype=torch.int32, device=dev()))
    def call():  # noqa: E306
        return idx.attention_fp8(q, k, v, s["ks"], s["vs"], bt.to(dev()), torch.tensor(lens, dtype=torch.int32, device=dev()),
                                 **more)
    base = call()
    bad = [(0, 2, 0), (1, 5, 1)]  # request, its block, K/V head; request 0's block 2 begins at position 64
    for b, j, h in bad:
        s[which][int(bt[b, j]), h] = value
    out = call()
    clean()
    assert not torch.isnan(base).any()
    per = H // Hkv
    for b in range(3):
        for t in range(n):
            extent = lens[b] - n + t + 1
            for h in range(Hkv):
                hit = any(bb == b and hh == h and extent > j * bs for bb, j, hh in bad)
                got = out[b, t, h * per:(h + 1) * per]
                assert torch.isnan(got).all() if hit else torch.equal(got, base[b, t, h * per:(h + 1) * per]), (b, t, h)


# ---- offsets past 32 bits ----------------------------------------------------------------------------

@pytest.mark.parametrize("D,bs", [(128, 64), (64, 32)])
def test_attention_selects_past_32_bits_of_a_pool(D, bs):
    """Selected rows that lie past 2^31 bytes of the pools: the bits of the same rows in small ones."""
    B, H, used = 3, 8, 24
    blocks = (1 << 31) // (bs * D) + used
    g = gen(81)
    k, v = (torch.randn(used, 1, bs, D, generator=g).mul(60).to(torch.float8_e4m3fn).to(dev()) for _ in range(2))
    ks, vs = ((torch.rand(used, 1, generator=g) * 0.02 + 0.01).to(dev()) for _ in range(2))
    bt = torch.randperm(used, generator=g).int().view(B, -1).to(dev())
    seq = torch.tensor([8 * bs, 5 * bs + 3, 1], dtype=torch.int32, device=dev())
    q = torch.randn(B, 1, H, D, generator=g).bfloat16().to(dev())
    cand = torch.stack([torch.randperm(8 * bs, generator=g)[:150] for _ in range(B)]).int()
    cand = torch.stack((cand, cand), -1).contiguous().to(dev())
    ranges = torch.tensor([[0] * B, [150] * B], dtype=torch.int32, device=dev())
    want = idx.attention_fp8(q, k, v, ks, vs, bt, seq, candidates=cand, ranges=ranges)
    big, first = [], blocks - used
    for t in (k, v):
        pool = torch.empty(blocks, 1, bs, D, dtype=torch.uint8, device=dev())
        pool[first:] = t.view(torch.uint8)
        big.append(pool.view(torch.float8_e4m3fn))
    for t in (ks, vs):
        big.append(torch.full((blocks, 1), math.nan, device=dev()))
        big[-1][first:] = t
    got = idx.attention_fp8(q, *big, bt + first, seq, candidates=cand, ranges=ranges)
    clean()
    assert (want[0] != 0).any() and torch.equal(got, want)


def test_attention_selects_past_32_bits_of_the_slots():
    B, H, D, bs, slots = 4096, 2, 64, 32, 70000   # 2.3 GB of slots
    g = gen(82)
    k, v = (torch.randn(4, 1, bs, D, generator=g).mul(60).to(torch.float8_e4m3fn).to(dev()) for _ in range(2))
    sc = torch.full((4, 1), 1.0 / 60, device=dev())
    bt = torch.randint(4, (B, 3), generator=g, dtype=torch.int32).to(dev())
    seq = torch.full((B,), 96, dtype=torch.int32, device=dev())
    q = torch.randn(B, 1, H, D, generator=g).bfloat16().to(dev())
    few = torch.randint(96, (B, 20, 2), generator=g, dtype=torch.int32).to(dev())
    few_ranges = torch.tensor([[0] * B, [20] * B], dtype=torch.int32, device=dev())
    want = idx.attention_fp8(q, k, v, sc, sc, bt, seq, candidates=few, ranges=few_ranges)
    wide = torch.full((B, slots, 2), -1, dtype=torch.int32, device=dev())
    wide[:, slots - 20:] = few
    got = idx.attention_fp8(q, k, v, sc, sc, bt, seq, candidates=wide, ranges=few_ranges + (slots - 20))
    clean()
    assert torch.equal(got, want)


# ---- refusals --------------------------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv", [(4, 8), (1, 2), (12, 8)])
def test_attention_refuses_heads_that_are_no_multiple(H, Hkv):
    D, bs = 64, 32
    pool = torch.zeros(2, Hkv, bs, D, dtype=torch.uint8, device=dev())
    sc = torch.ones(2, Hkv, device=dev())
    bt, sl = torch.zeros(2, 1, dtype=torch.int32, device=dev()), torch.ones(2, dtype=torch.int32, device=dev())
    with pytest.raises(idx.IdxError, match="multiple"):
        idx.attention_fp8(torch.zeros(2, 1, H, D, dtype=torch.bfloat16, device=dev()), pool, pool, sc, sc, bt, sl)

"""The 4-bit cache's writer and reader at the sizes where a warp takes several rounds of a token's heads, the
attention over it of queries that are not finite, and the cache under a layer that selects."""
import math

import numpy as np
import pytest
import torch

import heads_plain as plain4
import layer_plain as plain
import oracle
import paged_fp8_mqa_gb300 as idx
import test_cache4_gpu as small
import test_layer_example_gpu as serving

pytestmark = pytest.mark.gpu

DTYPES = small.DTYPES
dev, gen, clean = small.dev, small.gen, small.clean


def rounds(T, H, at_once, apart):
    """Whether a warp takes four rounds of at_once heads (keys and values `apart`, or one after the other)."""
    n = 2 * -(-H // at_once) if apart else -(-2 * H // at_once)
    return T * n > 16384


@pytest.mark.parametrize("H,D,bs,rot,offset,interleaved,name,layout", [
    (3, 128, 64, 64, 0, False, "bf16", "plain"),
    (5, 128, 32, 128, 0, True, "f16", "strided"),
    (9, 128, 64, 64, 32, False, "f32", "plain"),   # six rounds, the fourth of values beside three of keys
    (9, 64, 128, 0, 0, False, "bf16", "strided"),
    (3, 64, 32, 64, 0, False, "f32", "plain"),
    (17, 64, 64, 16, 8, True, "bf16", "plain"),
    (5, 128, 64, 20, 6, False, "bf16", "plain"),   # pairs that do not fill pieces: the general writer
    (3, 64, 32, 32, 0, False, "f16", "plain"),     # groups of 32 that four lanes' pieces are not: the same
    (9, 128, 128, 128, 0, False, "f32", "odd"),
    (3, 128, 64, 0, 0, False, "bf16", "odd"),
])
def test_long_runs_in_several_rounds_equal_their_parts(H, D, bs, rot, offset, interleaved, name, layout):
    """More tokens than make a warp take four rounds, against calls where it takes one: the same bytes, and the
    same rows read back."""
    clean()
    g = gen(H * 1000 + D)
    lens = [9000, 1, 7777]
    T, part = sum(lens), 600
    pieces = layout != "odd" and (rot == 0 or interleaved and rot % 8 == offset % 8 == 0 or rot % 64 == offset % 32 == 0)
    at_once = 512 // D if pieces else 256 // D
    assert rounds(T, H, at_once, pieces) and not rounds(part, H, at_once, pieces)
    reads = rounds(T, H, 512 // D, False)
    assert reads or H == 3 and D == 64  # (where two rounds hold all the heads)
    rows, blocks = small.pages_for(lens, bs, g)
    bt = torch.tensor(rows, dtype=torch.int32).to(dev())
    gap = dict(plain=0, strided=8, odd=3)[layout]
    k, v = (torch.randn(T, H, D + gap, generator=g).to(DTYPES[name]).to(dev())[:, :, :D] for _ in range(2))
    how = dict(table=idx.rotary_table(9000, rot) if rot else None, interleaved=interleaved, rot_offset=offset)
    whole, parts = small.empty_cache(blocks, H, bs, D, gen(1)), small.empty_cache(blocks, H, bs, D, gen(1))
    at = [0, *np.cumsum(lens).tolist()]
    starts = torch.tensor(at, dtype=torch.int32).to(dev())
    seq = torch.tensor(lens, dtype=torch.int32).to(dev())
    idx.kv_append_fp4(k, v, *whole, bt, seq, token_starts=starts, **how)
    back = idx.kv_read_fp4(*whole, bt, seq, starts, tokens=T, dtype=DTYPES[name])
    given = [torch.full((T + 4, H + 1, D + gap), 7.0, dtype=DTYPES[name], device=dev()) for _ in range(2)]
    inner = [t[:T, :H, :D] for t in given]
    idx.kv_read_fp4(*whole, bt, seq, starts, tokens=T, k_out=inner[0], v_out=inner[1])
    clean()
    for b, n in enumerate(lens):
        for first in range(0, n, part):
            m = min(part, n - first)
            mine = slice(at[b] + first, at[b] + first + m)
            end = torch.tensor([first + m], dtype=torch.int32).to(dev())
            idx.kv_append_fp4(k[mine], v[mine], *parts, bt[b:b + 1], end, **how)
            one = idx.kv_read_fp4(*parts, bt[b:b + 1], end, tokens=m, dtype=DTYPES[name])
            assert all(torch.equal(x[mine], y) and torch.equal(z[mine], y) for x, z, y in zip(back, inner, one))
    clean()
    assert all(torch.equal(x, y) for x, y in zip(whole, parts))
    for t in given:  # what lies around the given rows is as it was
        assert (t[T:] == 7).all() and (t[:, H:] == 7).all() and (t[:, :, D:] == 7).all()
    # Some tokens against the formats (the small calls are, in every layout).
    kp, vp, ks, vs = (small.u8(t) for t in whole)
    picked = [0, 1, 8999, 9000, 9001, T - 1]
    place = [(b, p) for b, n in enumerate(lens) for p in range(n)]
    x = k.float().cpu().numpy()[picked]
    if rot:
        x = plain4.rotate_f32(x, [place[t][1] for t in picked], how["table"].cpu().numpy(), interleaved, offset)
    vv = v.float().cpu().numpy()[picked]
    for i, t in enumerate(picked):
        page, slot = rows[place[t][0]][place[t][1] // bs], place[t][1] % bs
        small.check_rows(x[i], kp[page, :, slot], ks[page, :, slot],
                         vv[i] if name == "f32" else vv[i].astype(np.float64), vp[page, :, slot], vs[page, :, slot])


@pytest.mark.parametrize("H,Hkv,D,bs,name,n", [(8, 1, 128, 64, "bf16", 1), (16, 2, 64, 32, "bf16", 2),
                                               (24, 1, 128, 32, "f16", 2), (20, 1, 64, 64, "bf16", 4),
                                               (64, 1, 128, 128, "bf16", 1)])
@pytest.mark.parametrize("picked", [False, True])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_query_that_is_not_finite_makes_its_own_row_nan(H, Hkv, D, bs, name, n, picked, value):
    clean()
    lens = [300, 0, 700, 5]
    c = small.attention_case(lens, n, H, Hkv, D, bs, name, 77)
    more, which = {}, None
    if picked:
        cand, ranges, which = small.selections(c, 64, gen(3))
        more = dict(candidates=cand, ranges=ranges)
    base, base_lse = small.run_attention(c, **more)
    bad = dict(c, q=c["q"].clone())
    hit = torch.zeros(base.shape[:3], dtype=torch.bool)
    for b, t, h, d in ((0, 0, 3, 5), (0, n - 1, H - 1, D - 1), (1, 0, 0, 0), (2, n - 1, 1, 32)):
        bad["q"][b, t, h, d] = value
        hit[b, t, h] = True
    out, lse = small.run_attention(bad, **more)
    clean()
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()  # (sees nothing)
    hit[1] = False
    hit = hit.to(dev())
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert not torch.isnan(out[~hit]).any()
    # The other rows are as exact as they were (their references may have moved at another tile).
    out[hit], lse[hit] = base[hit], base_lse[hit]
    small.check_attention(c, out, lse, which)


def test_the_select_feeds_the_attention_over_the_4_bit_cache():
    """The serving example's layer with this cache and normalised heads: the select's own slots and ranges, in a
    captured step, against the attention over each row's exact top positions."""
    example = serving.example()

    class Layer(example.SparseLayer):
        def __init__(self, *args, **more):
            super().__init__(*args, **more)
            blocks, heads, block, dim = self.k_pool.shape
            self.cache = (*(torch.zeros(blocks, heads, block, dim // 2, dtype=torch.uint8, device=dev()) for _ in range(2)),
                          torch.zeros(blocks, heads, block, dim // 32, dtype=torch.uint8, device=dev()),
                          torch.zeros(blocks, heads, block, device=dev()))
            self.k_weight = torch.linspace(0.5, 1.5, dim, device=dev())

        def write(self, x, token_starts=None):
            _, k = idx.norm_rotary(x.new_empty(x.shape[0], 0, self.D), self.heads_of(x, "k"), None, self.k_weight)
            idx.kv_append_fp4(k, self.heads_of(x, "v"), *self.cache, self.tables, self.lens,
                              token_starts=token_starts, table=self.table)

        def attend(self, slots=None, ranges=None):
            return idx.attention_fp4(self.q, *self.cache, self.tables, self.lens, candidates=slots, ranges=ranges)[:, 0]

    example.SparseLayer = Layer
    clean()
    layer, out, _ = example.run(batch=3, prompt=300, steps=2, top_k=40, **serving.SIZES)
    clean()
    lens = layer.lens.tolist()
    top, cnt = oracle.topk(layer.logits.cpu(), layer.row_ends.cpu(), 40)
    picked = [top[b, :cnt[b]].tolist() for b in range(3)]
    assert all(len(p) == min(40, n) for p, n in zip(picked, lens))
    kp, vp, ks, vs = layer.cache
    k = plain4.keys4(small.u8(kp), small.u8(ks))
    v = plain4.values4(small.u8(vp)) * small.f64(vs)[..., None]
    one = np.ones(k.shape[:2])
    ref, _, mag, _ = plain.attention(small.f64(layer.q), k, v, one, one, layer.tables.cpu().numpy(), lens, 64,
                                     128 ** -0.5, picked)
    # Weights within 2^-10 of themselves, scores within 2^-10 here, the output rounded to 2^-8.
    lim = 2.0 ** -8 * mag[:, 0] + 2.0 ** -8 * np.abs(ref[:, 0]) + 2.0 ** -12
    assert (np.abs(small.f64(out) - ref[:, 0]) <= lim).all()
    # Selecting everything is attending everywhere.
    layer, out, _ = example.run(batch=3, prompt=200, steps=3, top_k=256, **serving.SIZES)
    dense = layer.attend()
    clean()
    lim = 2.0 ** -6 * dense.float().abs().amax(-1, keepdim=True) + 2.0 ** -7
    assert ((out.float() - dense.float()).abs() <= lim).all()

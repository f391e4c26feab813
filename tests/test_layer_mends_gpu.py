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

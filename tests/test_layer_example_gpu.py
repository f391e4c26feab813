"""The serving example runs every operator around the indexer together with the indexer."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import layer_plain as plain
import oracle
import paged_fp8_mqa_gb300 as idx

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_layer.py")


def example():
    spec = importlib.util.spec_from_file_location("sparse_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


SIZES = dict(hidden=256, heads=16, kv_heads=2, index_heads=64, rot=32)


def test_selecting_everything_is_attending_everywhere():
    idx.device_status(clear=True)
    layer, out, _ = example().run(batch=3, prompt=200, steps=3, top_k=256, **SIZES)
    dense = layer.attend()
    torch.cuda.synchronize()
    assert idx.device_status(clear=True) == 0
    assert layer.lens.tolist() == [200 - 97 * b % 200 + 4 for b in range(3)]
    # The same weights in another order: both are within 2^-8 of each weight's share, twice rounded.
    lim = 2.0 ** -6 * dense.float().abs().amax(-1, keepdim=True) + 2.0 ** -7
    assert ((out.float() - dense.float()).abs() <= lim).all()


def test_a_step_attends_the_top_k_of_its_logits():
    layer, out, _ = example().run(batch=3, prompt=300, steps=2, top_k=40, scaling="yarn", factor=4.0, **SIZES)
    torch.cuda.synchronize()
    lens = layer.lens.tolist()
    top, cnt = oracle.topk(layer.logits.cpu(), layer.row_ends.cpu(), 40)
    picked = [top[b, :cnt[b]].tolist() for b in range(3)]
    assert all(len(p) == min(40, n) for p, n in zip(picked, lens))
    e4 = lambda t: plain.E4M3[t.view(torch.uint8).cpu().numpy()]  # noqa: E731
    f64 = lambda t: t.cpu().double().numpy()  # noqa: E731
    ref, _, mag, _ = plain.attention(f64(layer.q), e4(layer.k_pool), e4(layer.v_pool), f64(layer.k_scales),
                                     f64(layer.v_scales), layer.tables.cpu().numpy(), lens, 64, 128 ** -0.5, picked)
    # Weights within 2^-8 of themselves, scores within 2^-10 here, the output rounded to 2^-8.
    lim = 2.0 ** -7 * mag[:, 0] + 2.0 ** -8 * np.abs(ref[:, 0]) + 2.0 ** -12
    assert (np.abs(f64(out) - ref[:, 0]) <= lim).all()

"""The operators around the indexer without a GPU: the rotary frequencies (host arithmetic) and what
the entry points refuse before they touch a device."""
import ctypes
import math

import pytest
import torch

import paged_fp8_mqa_gb300 as idx

P = ctypes.c_void_p
FAKE = P(1 << 20)      # aligned and non-NULL: never dereferenced on these paths
ODD = P((1 << 20) + 2)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_fp8_mqa_gb300 import build
    if not idx.LIB_PATH.exists():
        build.build()
    return idx.lib()


def frequencies(rot, base=10000.0, scaling=0, factor=1.0, original=0.0, fast=32.0, slow=1.0):
    f, m = (ctypes.c_double * max(1, rot // 2))(), ctypes.c_double()
    st = idx.idx_rotary_frequencies(rot, base, scaling, factor, original, fast, slow, f, ctypes.byref(m))
    return st, list(f), m.value


def close(a, b):
    # A power and a few products in 64 bits.
    return all(abs(x - y) <= 1e-14 * abs(y) for x, y in zip(a, b)) and len(a) == len(b)


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 1024])
def test_frequencies_without_scaling_and_linear(rot):
    plain = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    st, f, m = frequencies(rot)
    assert st == 0 and m == 1.0 and close(f, plain)
    st, f, m = frequencies(rot, scaling=idx.IDX_ROTARY_LINEAR, factor=8.0)
    assert st == 0 and m == 1.0 and close(f, [x / 8 for x in plain])


@pytest.mark.parametrize("rot", [4, 64])
def test_frequencies_ntk(rot):
    """The base grows so that the slowest pair is slowed by exactly the factor."""
    st, f, m = frequencies(rot, scaling=idx.IDX_ROTARY_NTK, factor=4.0)
    _, plain, _ = frequencies(rot)
    assert st == 0 and m == 1.0
    assert f[0] == 1.0 and abs(f[-1] * 4.0 / plain[-1] - 1) <= 1e-13
    assert close(f, [(10000.0 * 4.0 ** (rot / (rot - 2))) ** (-2 * i / rot) for i in range(rot // 2)])


@pytest.mark.parametrize("rot,factor,original", [(64, 16.0, 4096.0), (128, 4.0, 32768.0), (32, 2.0, 50.0)])
def test_frequencies_by_parts(rot, factor, original):
    """Pairs that turn 32 times over the original positions stay, those that turn once at most are
    divided, the ramp between is linear in the pair's number."""
    st, f, m = frequencies(rot, scaling=idx.IDX_ROTARY_YARN, factor=factor, original=original)
    assert st == 0 and abs(m - (0.1 * math.log(factor) + 1)) <= 1e-15
    _, plain, _ = frequencies(rot)
    # turns(i) = original * plain[i] / (2 pi); the pair with `b` turns, in real numbers:
    at = lambda b: rot / 2 * math.log(original / (2 * math.pi * b)) / math.log(10000.0)  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    for i in range(rot // 2):
        turns = original * plain[i] / (2 * math.pi)
        if turns >= 32 and i <= lo:
            assert f[i] == plain[i]
        if turns <= 1 and i >= hi:
            assert abs(f[i] * factor / plain[i] - 1) <= 1e-14
        r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        assert abs(f[i] - plain[i] * (1 - r + r / factor)) <= 1e-14 * plain[i]


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=3), dict(rot=-2), dict(rot=1026), dict(rot=64, base=1.0),
    dict(rot=64, base=math.inf), dict(rot=64, base=math.nan), dict(rot=64, scaling=4),
    dict(rot=64, scaling=-1), dict(rot=64, scaling=1, factor=0.5), dict(rot=64, scaling=1, factor=math.nan),
    dict(rot=2, scaling=2, factor=2.0), dict(rot=64, scaling=3, factor=2.0),
    dict(rot=64, scaling=3, factor=2.0, original=100.0, fast=0.5, slow=1.0),
])
def test_frequencies_refused(kw):
    assert frequencies(**kw)[0] == idx.IDX_INVALID_ARG
    assert idx.idx_last_error()


def call(f, args, over):
    a = dict(args)
    assert set(over) <= set(a)
    a.update(over)
    return f(*a.values())


ROTARY = dict(x=FAKE, x_token=256, x_head=128, positions=FAKE, tokens=4, heads=2, dim=128,
              dtype=idx.IDX_DTYPE_BF16, table=FAKE, max_positions=100, rot=64, offset=0,
              interleaved=0, inverse=0, out=FAKE, out_token=256, out_head=128, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), 1), (dict(positions=None), 1), (dict(table=None), 1), (dict(out=None), 1),
    (dict(dtype=7), 2), (dict(tokens=-1), 1), (dict(heads=-1), 1), (dict(dim=0), 1),
    (dict(rot=63), 1), (dict(rot=0), 1), (dict(rot=130), 1), (dict(offset=65), 1), (dict(offset=-2), 1),
    (dict(max_positions=0), 1), (dict(x=P((1 << 20) + 1)), 1), (dict(table=P((1 << 20) + 4)), 1),
    (dict(tokens=0), 0), (dict(heads=0), 0),
])
def test_rotary_refused(over, code):
    assert call(idx.idx_rotary, ROTARY, over) == code, idx.idx_last_error()


def test_rotary_table_refused():
    f = (ctypes.c_double * 4)()
    assert idx.idx_rotary_table(None, 1.0, 8, 8, FAKE, None) == idx.IDX_INVALID_ARG
    assert idx.idx_rotary_table(f, 1.0, 8, 8, None, None) == idx.IDX_INVALID_ARG
    assert idx.idx_rotary_table(f, 1.0, -1, 8, FAKE, None) == idx.IDX_INVALID_ARG
    assert idx.idx_rotary_table(f, 1.0, 8, 7, FAKE, None) == idx.IDX_INVALID_ARG
    assert idx.idx_rotary_table(f, 1.0, 0, 8, FAKE, None) == idx.IDX_OK


TOKENS = dict(token_starts=None, seq_lens=FAKE, seq_stride=1, batch=2, next_n=2, tables=FAKE,
              table_stride=16, width=16, block_size=64, num_blocks=10)
PLACES = [
    (dict(seq_lens=None), 1), (dict(tables=None), 1), (dict(tokens=5), 1), (dict(tokens=-4), 1),
    (dict(next_n=0), 1), (dict(batch=-1), 1), (dict(table_stride=8), 1), (dict(seq_stride=0), 1),
    (dict(num_blocks=0), 1), (dict(block_size=48), 2), (dict(block_size=256), 2),
    (dict(batch=5000, tokens=10000), 2), (dict(dim=96), 2), (dict(dtype=3), 2), (dict(rot=200), 1),
    (dict(offset=100), 1), (dict(seq_lens=ODD), 1), (dict(token_starts=ODD), 1),
    (dict(batch=0, tokens=0), 0),
]
INDEX = dict(k=FAKE, k_token=128, q=FAKE, q_token=1024, q_head=128, weights=FAKE, w_token=8,
             dtype=idx.IDX_DTYPE_BF16, tokens=4, heads=8, dim=128, table=FAKE, max_positions=100,
             rot=64, offset=0, interleaved=0, **TOKENS, pool=FAKE, q_out=FAKE, w_out=FAKE, stream=None)
APPEND = dict(k=FAKE, k_token=1024, k_head=128, v=FAKE, v_token=1024, v_head=128,
              dtype=idx.IDX_DTYPE_BF16, tokens=4, heads=8, dim=128, table=FAKE, max_positions=100,
              rot=64, offset=0, interleaved=0, **TOKENS, k_pool=FAKE, v_pool=FAKE, k_scales=FAKE,
              v_scales=FAKE, stream=None)


@pytest.mark.parametrize("over,code", PLACES + [
    (dict(k=None), 1), (dict(pool=None), 1), (dict(q_out=None), 1), (dict(w_out=None), 1),
    (dict(weights=None), 1), (dict(heads=0), 1), (dict(pool=P((1 << 20) + 8)), 1),
])
def test_index_prepare_refused(over, code):
    assert call(idx.idx_index_prepare, INDEX, over) == code, idx.idx_last_error()


@pytest.mark.parametrize("over,code", PLACES + [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k_pool=None), 1), (dict(v_scales=None), 1),
    (dict(heads=0), 1), (dict(dim=192), 2), (dict(v_pool=P((1 << 20) + 8)), 1), (dict(k=P((1 << 20) + 1)), 1),
])
def test_kv_append_refused(over, code):
    assert call(idx.idx_kv_append, APPEND, over) == code, idx.idx_last_error()


ATTENTION = dict(q=FAKE, q_batch=8192, q_token=8192, q_head=128, dtype=idx.IDX_DTYPE_BF16, k_pool=FAKE,
                 v_pool=FAKE, k_scales=FAKE, v_scales=FAKE, num_blocks=10, block_size=64, tables=FAKE,
                 table_stride=16, width=16, seq_lens=FAKE, seq_stride=1, batch=2, next_n=1, heads=64,
                 kv_heads=8, dim=128, scale=0.1, candidates=None, slots=0, ranges=None, num_sms=4,
                 out=FAKE, lse=None, workspace=FAKE, workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(k_scales=None), 1), (dict(tables=None), 1),
    (dict(batch=-1), 1), (dict(num_blocks=0), 1), (dict(table_stride=8), 1), (dict(seq_stride=0), 1),
    (dict(heads=60), 1), (dict(kv_heads=0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1),
    (dict(candidates=FAKE), 1), (dict(candidates=FAKE, ranges=FAKE), 1), (dict(q=P((1 << 20) + 8)), 1),
    (dict(q_head=100), 1), (dict(q_token=8196), 1), (dict(num_sms=-1), 1), (dict(num_sms=2000), 1),
    (dict(workspace=None), 1), (dict(workspace_bytes=100), 1), (dict(workspace=P((1 << 20) + 16)), 1),
    (dict(num_blocks=1 << 24), 1), (dict(dtype=idx.IDX_DTYPE_F32), 2), (dict(next_n=5), 2),
    (dict(batch=5000), 2), (dict(dim=192), 2), (dict(block_size=16), 2), (dict(heads=8192), 2),
    (dict(batch=0), 0),
])
def test_attention_refused(over, code):
    assert call(idx.idx_attention_fp8, ATTENTION, over) == code, idx.idx_last_error()


def test_attention_workspace_size():
    f = idx.idx_attention_workspace_bytes
    assert f(-1, 1, 8, 1, 128, 152) == -1 and f(1, 0, 8, 1, 128, 152) == -1 and f(1, 1, 8, 0, 128, 152) == -1
    # Two partial results of the largest row tile (here 64 rows of dim + 2 floats) for each CTA at least.
    assert f(4, 1, 64, 1, 128, 152) >= 2 * 152 * 64 * 130 * 4
    assert f(4, 1, 64, 1, 128, 152) < f(4, 1, 64, 1, 128, 300)
    assert f(0, 1, 8, 1, 64, 1) > 0


def test_host_tensors_and_shapes_are_refused():
    bf, i32 = torch.bfloat16, torch.int32
    x = torch.zeros(4, 2, 64, dtype=bf)
    pool = torch.zeros(2, 2, 32, 64, dtype=torch.uint8)
    sc, bt, sl = torch.zeros(2, 2), torch.zeros(4, 1, dtype=i32), torch.ones(4, dtype=i32)
    for f in (lambda: idx.rotary(x, torch.zeros(4, dtype=i32), torch.zeros(8, 32, 2)),
              lambda: idx.rotary([1], None, None),
              lambda: idx.index_prepare(x[:, 0], torch.zeros(2, 32 * 68, dtype=torch.uint8), bt, sl),
              lambda: idx.kv_append(x, x, pool, pool, sc, sc, bt, sl),
              lambda: idx.attention_fp8(x[:, None], pool, pool, sc, sc, bt, sl),
              lambda: idx.attention_fp8(None, pool, pool, sc, sc, bt, sl)):
        with pytest.raises(TypeError, match="CUDA"):
            f()
    with pytest.raises(ValueError, match="scaling"):
        idx.rotary_table(8, 4, scaling="other")

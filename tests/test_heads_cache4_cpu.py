"""What the entry points of the normalised heads and of the 4-bit cache refuse before they touch a
device, and the axes' host arithmetic."""
import ctypes
import math

import pytest
import torch

import heads_plain as plain4
import paged_fp8_mqa_gb300 as idx

P = ctypes.c_void_p
FAKE = P(1 << 20)      # aligned and non-NULL: never dereferenced on these paths
ODD = P((1 << 20) + 2)
AXES = (ctypes.c_uint8 * 512)(*[i % 3 for i in range(512)])


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_fp8_mqa_gb300 import build
    if not idx.LIB_PATH.exists():
        build.build()
    return idx.lib()


def call(f, args, over):
    a = dict(args)
    assert set(over) <= set(a)
    a.update(over)
    return f(*a.values())


def test_axes_of_pairs():
    assert idx.rotary_axes((2, 3)) == (0, 0, 1, 1, 1)
    assert idx.rotary_axes((2, 4, 1), in_turn=True) == (0, 1, 2, 0, 1, 1, 1)
    assert idx.rotary_axes((3,)) == (0, 0, 0) and idx.rotary_axes((0, 2)) == (1, 1)
    for bad in ((), (1, 1, 1, 1, 1), (-1, 2)):
        with pytest.raises(ValueError, match="sections"):
            idx.rotary_axes(bad)
    from paged_fp8_mqa_gb300.heads import _axis_bytes
    assert list(_axis_bytes((0, 2, 1), 3, 3)) == [0, 2, 1]
    for axes, count, pairs in (((0, 1), 2, 3), ((0, 1, 2), 2, 3), ((0, -1, 1), 2, 3), ((0, 1.0, 1), 2, 3)):
        with pytest.raises(ValueError, match="axes"):
            _axis_bytes(axes, count, pairs)


def test_the_plain_codes():
    """The formats' tables, and the rounding at every border."""
    assert plain4.E2M1[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and plain4.E2M1[9] == -0.5
    assert plain4.e2m1(plain4.BORDERS).tolist() == [0, 1, 1, 2, 2, 4, 4]
    assert plain4.e2m1([7.0, -9.0, 0.26, -0.24]).tolist() == [6, -6, 0.5, 0]
    assert plain4.ue8m0([0, 127, 254]).tolist() == [2.0 ** -127, 1, 2.0 ** 127] and math.isnan(plain4.ue8m0(255))
    assert [plain4.key_scale(x) for x in (6.0, 6.01, 3.0, 0.0)] == [0, 1, -1, -100]


TURN = dict(positions=FAKE, axis_stride=4, pair_axis=AXES, axes=3, table=FAKE, max_positions=100, rot=64,
            offset=0, interleaved=0)
TURNS = [
    (dict(rot=63), 1), (dict(rot=0), 1), (dict(rot=130), 1), (dict(offset=65), 1), (dict(offset=-2), 1),
    (dict(max_positions=0), 1), (dict(table=P((1 << 20) + 4)), 1), (dict(positions=None), 1),
    (dict(positions=ODD), 1), (dict(axes=0), 1), (dict(axes=5), 1), (dict(pair_axis=None), 1),
    (dict(axis_stride=-1), 1), (dict(axes=2), 1),  # (pairs of a third axis)
    (dict(dtype=7), 2), (dict(dim=0), 1), (dict(dim=1025), 2), (dict(tokens=-1), 1), (dict(tokens=0), 0),
]
ROTARY = dict(x=FAKE, x_token=256, x_head=128, positions=FAKE, axis_stride=4, pair_axis=AXES, axes=3,
              tokens=4, heads=2, dim=128, dtype=idx.IDX_DTYPE_BF16, table=FAKE, max_positions=100, rot=64,
              offset=0, interleaved=0, inverse=0, out=FAKE, out_token=256, out_head=128, stream=None)


@pytest.mark.parametrize("over,code", TURNS + [
    (dict(x=None), 1), (dict(out=None), 1), (dict(table=None), 1), (dict(heads=-1), 1), (dict(heads=0), 0),
    (dict(x=P((1 << 20) + 1)), 1), (dict(out=P((1 << 20) + 1)), 1),
])
def test_rotary_by_axes_refused(over, code):
    assert call(idx.idx_rotary_axes, ROTARY, over) == code, idx.idx_last_error()


NORM = dict(q=FAKE, q_token=256, q_head=128, heads=2, k=FAKE, k_token=128, k_head=128, kv_heads=1,
            dtype=idx.IDX_DTYPE_BF16, tokens=4, dim=128, q_weight=FAKE, k_weight=FAKE,
            weight_dtype=idx.IDX_DTYPE_BF16, eps=1e-6, **TURN)
NORMS = TURNS + [
    (dict(q=None), 1), (dict(k=None), 1), (dict(heads=-1), 1), (dict(kv_heads=-1), 1), (dict(eps=-1.0), 1),
    (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(weight_dtype=idx.IDX_DTYPE_F16), 2),
    (dict(weight_dtype=9), 2), (dict(q_weight=P((1 << 20) + 1)), 1),
    (dict(weight_dtype=idx.IDX_DTYPE_F32, k_weight=ODD), 1), (dict(q=P((1 << 20) + 1)), 1),
    (dict(k=P((1 << 20) + 1)), 1),
]


@pytest.mark.parametrize("over,code", NORMS + [
    (dict(q_out=None), 1), (dict(k_out=None), 1), (dict(k_out=P((1 << 20) + 1)), 1),
    (dict(heads=0, kv_heads=0), 0), (dict(table=None, positions=None, pair_axis=None, axes=9, tokens=0), 0),
])
def test_norm_rotary_refused(over, code):
    args = dict(NORM, q_out=FAKE, qo_token=256, qo_head=128, k_out=FAKE, ko_token=128, ko_head=128, stream=None)
    assert call(idx.idx_norm_rotary, args, over) == code, idx.idx_last_error()


@pytest.mark.parametrize("over,code", [x for x in NORMS if x[1]] + [
    (dict(gq=None), 1), (dict(gk=None), 1), (dict(dq=None), 1), (dict(dk=None), 1),
    (dict(q_weight=None), 1), (dict(k_weight=None), 1), (dict(dqw=P((1 << 20) + 1)), 1),
])
def test_norm_rotary_backward_refused(over, code):
    args = dict(NORM, gq=FAKE, gq_token=256, gq_head=128, gk=FAKE, gk_token=128, gk_head=128, dq=FAKE,
                dk=FAKE, dqw=FAKE, dkw=FAKE, workspace=FAKE, workspace_bytes=1 << 30, stream=None)
    assert call(idx.idx_norm_rotary_backward, args, over) == code, idx.idx_last_error()


@pytest.mark.parametrize("weight_dtype", [0, 3, 9, -1, 1 << 30])
def test_without_weights_their_dtype_is_not_read(weight_dtype):
    """No weights: any weight_dtype is accepted (nothing is launched without tokens)."""
    over = dict(q_weight=None, k_weight=None, weight_dtype=weight_dtype)
    args = dict(NORM, q_out=FAKE, qo_token=256, qo_head=128, k_out=FAKE, ko_token=128, ko_head=128, stream=None)
    assert call(idx.idx_norm_rotary, args, dict(over, tokens=0)) == 0, idx.idx_last_error()
    args = dict(NORM, gq=FAKE, gq_token=256, gq_head=128, gk=FAKE, gk_token=128, gk_head=128, dq=FAKE,
                dk=FAKE, dqw=None, dkw=None, workspace=None, workspace_bytes=0, stream=None)
    # (Refused for the workspace, or where there is no device, after the weights have been looked at.)
    assert call(idx.idx_norm_rotary_backward, args, over) in (1, 3), idx.idx_last_error()


def test_norm_rotary_workspace_refused():
    assert idx.idx_norm_rotary_workspace_bytes(0) == -1 and idx.idx_norm_rotary_workspace_bytes(1025) == -1


PLACE = dict(token_starts=None, seq_lens=FAKE, seq_stride=1, batch=2, next_n=2, tables=FAKE,
             table_stride=16, width=16, block_size=64, num_blocks=10)
PLACES = [
    (dict(seq_lens=None), 1), (dict(tables=None), 1), (dict(tokens=5), 1), (dict(tokens=-4), 1),
    (dict(next_n=0), 1), (dict(batch=-1), 1), (dict(table_stride=8), 1), (dict(seq_stride=0), 1),
    (dict(num_blocks=0), 1), (dict(block_size=48), 2), (dict(batch=5000, tokens=10000), 2),
    (dict(dim=96), 2), (dict(dim=192), 2), (dict(dtype=3), 2), (dict(seq_lens=ODD), 1),
    (dict(token_starts=ODD), 1), (dict(batch=0, tokens=0), 0), (dict(heads=0), 1),
    (dict(k_pool=None), 1), (dict(v_pool=None), 1), (dict(k_scales=None), 1), (dict(v_scales=None), 1),
    (dict(v_pool=P((1 << 20) + 8)), 1), (dict(v_scales=ODD), 1), (dict(k=P((1 << 20) + 1)), 1),
    (dict(v=None), 1),
]
POOLS = dict(k_pool=FAKE, v_pool=FAKE, k_scales=FAKE, v_scales=FAKE)


@pytest.mark.parametrize("over,code", PLACES + [(dict(rot=200), 1), (dict(offset=100), 1)])
def test_kv_append_fp4_refused(over, code):
    args = dict(k=FAKE, k_token=1024, k_head=128, v=FAKE, v_token=1024, v_head=128,
                dtype=idx.IDX_DTYPE_BF16, tokens=4, heads=8, dim=128, table=FAKE, max_positions=100,
                rot=64, offset=0, interleaved=0, **PLACE, **POOLS, stream=None)
    assert call(idx.idx_kv_append_fp4, args, over) == code, idx.idx_last_error()


@pytest.mark.parametrize("over,code", PLACES + [(dict(batch=0, token_starts=FAKE), 1)])
def test_kv_read_fp4_refused(over, code):
    args = dict(**POOLS, num_blocks=10, block_size=64, heads=8, dim=128, token_starts=None, tokens=4,
                seq_lens=FAKE, seq_stride=1, batch=2, next_n=2, tables=FAKE, table_stride=16, width=16,
                clear=1, dtype=idx.IDX_DTYPE_BF16, k=FAKE, k_token=1024, k_head=128, v=FAKE, v_token=1024,
                v_head=128, stream=None)
    assert call(idx.idx_kv_read_fp4, args, over) == code, idx.idx_last_error()


ATTENTION = dict(q=FAKE, q_batch=8192, q_token=8192, q_head=128, dtype=idx.IDX_DTYPE_BF16, k_pool=FAKE,
                 v_pool=FAKE, k_scales=FAKE, v_scales=FAKE, num_blocks=10, block_size=64, tables=FAKE,
                 table_stride=16, width=16, seq_lens=FAKE, seq_stride=1, batch=2, next_n=1, heads=64,
                 kv_heads=8, dim=128, scale=0.1, candidates=None, slots=0, ranges=None, num_sms=4,
                 out=FAKE, lse=None, workspace=FAKE, workspace_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(k_scales=None), 1), (dict(tables=None), 1),
    (dict(batch=-1), 1), (dict(num_blocks=0), 1), (dict(heads=60), 1), (dict(kv_heads=0), 1),
    (dict(scale=math.inf), 1), (dict(candidates=FAKE), 1), (dict(q=P((1 << 20) + 8)), 1), (dict(q_head=100), 1),
    (dict(k_pool=P((1 << 20) + 16)), 1), (dict(v_pool=P((1 << 20) + 16)), 1),
    (dict(k_scales=P((1 << 20) + 8)), 1), (dict(v_scales=P((1 << 20) + 4)), 1),
    (dict(workspace=None), 1), (dict(workspace_bytes=100), 1), (dict(num_blocks=1 << 24), 1),
    (dict(dtype=idx.IDX_DTYPE_F32), 2), (dict(next_n=5), 2), (dict(batch=5000), 2), (dict(dim=192), 2),
    (dict(block_size=16), 2), (dict(heads=8192), 2), (dict(batch=0), 0),
])
def test_attention_fp4_refused(over, code):
    assert call(idx.idx_attention_fp4, ATTENTION, over) == code, idx.idx_last_error()


def test_host_tensors_are_refused():
    bf, i32 = torch.bfloat16, torch.int32
    x = torch.zeros(4, 2, 64, dtype=bf)
    cache = (torch.zeros(2, 2, 32, 32, dtype=torch.uint8), torch.zeros(2, 2, 32, 32, dtype=torch.uint8),
             torch.zeros(2, 2, 32, 2, dtype=torch.uint8), torch.zeros(2, 2, 32))
    bt, sl = torch.zeros(4, 1, dtype=i32), torch.ones(4, dtype=i32)
    for f in (lambda: idx.rotary(x, torch.zeros(2, 4, dtype=i32), torch.zeros(8, 32, 2), axes=[0, 1] * 16),
              lambda: idx.norm_rotary(x, x), lambda: idx.norm_rotary(None, x),
              lambda: idx.kv_append_fp4(x, x, *cache, bt, sl),
              lambda: idx.kv_read_fp4(*cache, bt, sl, tokens=4),
              lambda: idx.attention_fp4(x[:, None], *cache, bt, sl)):
        with pytest.raises(TypeError, match="CUDA"):
            f()


@pytest.mark.parametrize("call", ["axes", "norm", "append", "read", "attention"])
@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_their_tensors_device(call, current, monkeypatch):
    """Tensors said to be on device 1, with device 0 or 1 current: every C call is made with 1 current."""
    from paged_fp8_mqa_gb300 import cache4, heads, layer
    now, entered, seen = [current], [], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index
            entered.append(self.index)

        def __exit__(self, *_):
            now[0] = self.before

    def c_call(*_):
        seen.append(now[0])
        return 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    for module in (layer, heads, cache4):
        monkeypatch.setattr(module, "_index", lambda t, name: 1)
        monkeypatch.setattr(module, "_on", lambda *a: 0)
    monkeypatch.setattr(layer, "_sizes", {})
    monkeypatch.setattr(layer, "idx_attention_workspace_bytes", c_call)
    for module, name in ((heads, "idx_rotary_axes"), (heads, "idx_norm_rotary"), (cache4, "idx_kv_append_fp4"),
                         (cache4, "idx_kv_read_fp4"), (cache4, "idx_attention_fp4")):
        monkeypatch.setattr(module, name, c_call)
    i32 = torch.int32
    x, table = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(8, 32, 2)
    pos, bt, sl = torch.zeros(2, 2, dtype=i32), torch.zeros(2, 1, dtype=i32), torch.ones(2, dtype=i32)
    cache = (torch.zeros(2, 4, 32, 32, dtype=torch.uint8), torch.zeros(2, 4, 32, 32, dtype=torch.uint8),
             torch.zeros(2, 4, 32, 2, dtype=torch.uint8), torch.zeros(2, 4, 32))
    {"axes": lambda: idx.rotary(x, pos, table, axes=[0, 1] * 16),
     "norm": lambda: idx.norm_rotary(x, x, None, None, pos, table, axes=[0, 1] * 16),
     "append": lambda: idx.kv_append_fp4(x, x, *cache, bt, sl),
     "read": lambda: idx.kv_read_fp4(*cache, bt, sl, tokens=2),
     "attention": lambda: idx.attention_fp4(x[:, None], *cache, bt, sl)}[call]()
    assert seen == [1] * (2 if call == "attention" else 1)
    assert entered == ([1] if current == 0 else []) and now == [current]

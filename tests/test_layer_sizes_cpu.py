"""The operators around the indexer without a GPU: sizes that they refuse, the device that they run on,
the arithmetic of their split."""
import bisect
import random
import shutil
import subprocess

import pytest
import torch

import paged_fp8_mqa_gb300 as idx
from paged_fp8_mqa_gb300 import layer


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_fp8_mqa_gb300 import build
    if not idx.LIB_PATH.exists():
        build.build()
    return idx.lib()


@pytest.mark.parametrize("batch,next_n,heads,kv_heads,dim,sms", [
    (2, 1, 4, 8, 128, 4),        # fewer query heads than K/V heads
    (2, 1, 1, 2, 64, 4), (2, 1, 12, 8, 128, 4), (2, 5, 8, 8, 128, 4), (4097, 1, 8, 8, 128, 4),
    (2, 1, 8192, 8, 128, 4), (2, 1, 8, 8, 192, 4), (2, 2 ** 31 - 1, 64, 1, 128, 4), (2, 1, 8, 8, 128, 1025),
    (2, 1, 8, 8, 128, -1),
])
def test_attention_workspace_of_refused_sizes(batch, next_n, heads, kv_heads, dim, sms):
    assert idx.idx_attention_workspace_bytes(batch, next_n, heads, kv_heads, dim, sms) == -1


@pytest.mark.parametrize("call", ["rotary", "index_prepare", "kv_append", "attention_fp8", "keyword"])
@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_their_tensors_device(call, current, monkeypatch):
    """Tensors said to be on device 1, with device 0 or 1 current: every C call is made with 1 current."""
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
    monkeypatch.setattr(layer, "_index", lambda t, name: 1)
    monkeypatch.setattr(layer, "_on", lambda *a: 0)
    monkeypatch.setattr(layer, "_sizes", {})
    for name in ("idx_rotary", "idx_index_prepare", "idx_kv_append", "idx_attention_fp8",
                 "idx_attention_workspace_bytes"):
        monkeypatch.setattr(layer, name, c_call)
    i32 = torch.int32
    x, pos = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=i32)
    table, bt, sl = torch.zeros(8, 32, 2), torch.zeros(2, 1, dtype=i32), torch.ones(2, dtype=i32)
    pool, sc = torch.zeros(2, 4, 32, 64, dtype=torch.uint8), torch.ones(2, 4)
    {"rotary": lambda: idx.rotary(x, pos, table),
     "keyword": lambda: idx.rotary(x=x, positions=pos, table=table),
     "index_prepare": lambda: idx.index_prepare(x[:, 0], torch.zeros(2, 32 * 68, dtype=torch.uint8), bt, sl),
     "kv_append": lambda: idx.kv_append(x, x, pool, pool, sc, sc, bt, sl),
     "attention_fp8": lambda: idx.attention_fp8(x[:, None], pool, pool, sc, sc, bt, sl)}[call]()
    assert seen == [1] * (2 if call == "attention_fp8" else 1)
    assert entered == ([1] if current == 0 else []) and now == [current]


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_runs_of_a_line(tmp_path):
    """The split's two formulas against whole numbers without a limit, also for lines of more than 2^31
    items, the first runs of them among others."""
    (tmp_path / "runs.cpp").write_text("""
#include <cstdio>
#include "runs.h"
int main() {
  long long total, runs, c, x;
  while (scanf("%lld %lld %lld %lld", &total, &runs, &c, &x) == 4)
    printf("%lld %lld\\n", (long long)idx::run_begin(total, runs, c), (long long)idx::run_of(total, runs, x));
}
""")
    csrc = idx.LIB_PATH.parent / "csrc"
    subprocess.run(["g++", "-O1", f"-I{csrc}", "-o", str(tmp_path / "runs"), str(tmp_path / "runs.cpp")], check=True)
    rng, cases = random.Random(5), []
    for total in (1, 2, 127, 304, 305, 4097, (1 << 21) - 1, 1 << 21, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 1, 3 << 30,
                  2 ** 32 - 1, 2 ** 32 + 7, 2 ** 40, 2 ** 48):
        for runs in (1, 2, 151, 304, 2048):
            if runs > total:
                continue
            for _ in range(20):
                c = rng.choice([0, 1, runs - 1, runs, rng.randint(0, runs)])
                x = rng.choice([0, total - 1, total * min(c, runs - 1) // runs + rng.randint(-1, 1),
                                rng.randrange(total), rng.randrange(min(total, 1 << 22))])
                cases.append((total, runs, c, min(max(x, 0), total - 1)))
    run = subprocess.run([str(tmp_path / "runs")], input="\n".join("%d %d %d %d" % c for c in cases), text=True,
                         capture_output=True)
    assert run.returncode == 0, run.returncode
    for (total, runs, c, x), line in zip(cases, run.stdout.split("\n")):
        begins = [total * i // runs for i in range(runs)]
        assert line == f"{total * c // runs} {bisect.bisect_right(begins, x) - 1}", (total, runs, c, x, line)

"""One sparse-attention layer served with this library: prompts fill the indexer's pool and the K/V
cache, then each decode step rotates, writes, scores, selects and attends, captured in one CUDA
graph and replayed.

    python examples/sparse_layer.py [--batch 8] [--prompt 6000] [--steps 32] [--top-k 2048]

The weights are random; the projections are plain matrix products.  With top_k at least the context's
length the selection is everything, and the step's output is checked against the attention over
every position.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import paged_fp8_mqa_gb300 as idx  # noqa: E402


class SparseLayer:
    """A layer of `heads` query heads over `kv_heads` K/V heads and an indexer of `index_heads`
    heads, with its caches: pages of `block` tokens, one table for both pools."""

    def __init__(self, batch, max_len, *, hidden=1024, heads=64, kv_heads=8, index_heads=64, dim=128,
                 block=64, rot=64, top_k=2048, scaling="none", factor=1.0, seed=0):
        dev = torch.device("cuda")
        g = torch.Generator(dev).manual_seed(seed)
        self.B, self.H, self.Hkv, self.Hi, self.D = batch, heads, kv_heads, index_heads, dim
        self.top_k, self.max_len = top_k, max_len
        pages = -(-max_len // block)
        self.tables = torch.randperm(batch * pages, generator=g, device=dev).int().view(batch, pages)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.index_pool = torch.zeros(batch * pages, block * (dim + 4), dtype=torch.uint8, device=dev)
        shape = (batch * pages, kv_heads, block, dim)
        self.k_pool, self.v_pool = (torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev)
                                    for _ in range(2))
        self.k_scales, self.v_scales = (torch.zeros(shape[:2], device=dev) for _ in range(2))
        self.table = idx.rotary_table(max_len, rot, scaling=scaling, factor=factor,
                                      original_positions=max_len / factor)
        sizes = dict(q=heads * dim, k=kv_heads * dim, v=kv_heads * dim, iq=index_heads * dim, ik=dim,
                     iw=index_heads)
        self.w = {n: (torch.randn(hidden, m, generator=g, device=dev) * hidden ** -0.5).bfloat16()
                  for n, m in sizes.items()}
        # The select's buffers: thresholds of +inf ask for each row's exact top_k.
        self.logits = torch.empty(batch, idx.idx_padded_seq_len(max_len), device=dev)
        self.row_ends = torch.empty(batch, dtype=torch.int32, device=dev)
        self.thresholds = torch.empty(batch, device=dev)
        self.counters = torch.empty(batch, 2, dtype=torch.int32, device=dev)
        self.slots = torch.empty(batch, 2 * top_k - 1, 2, dtype=torch.int32, device=dev)
        self.arrivals = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.ranges = torch.empty(2, batch, dtype=torch.int32, device=dev)

    def heads_of(self, x, name):
        return (x @ self.w[name]).view(x.shape[0], -1, self.D)

    def write(self, x, token_starts=None):
        """The new tokens' keys and values into both pools (lens counts them already)."""
        idx.kv_append(self.heads_of(x, "k"), self.heads_of(x, "v"), self.k_pool, self.v_pool,
                      self.k_scales, self.v_scales, self.tables, self.lens,
                      token_starts=token_starts, table=self.table)

    def prompt(self, x, lens):
        """Prompts of the given lengths (rows of x, request by request) into empty caches."""
        starts = torch.zeros(self.B + 1, dtype=torch.int32, device=x.device)
        starts[1:] = torch.cumsum(lens, 0)
        self.lens.copy_(lens)
        idx.index_prepare(x @ self.w["ik"], self.index_pool, self.tables, self.lens,
                          token_starts=starts, table=self.table)
        self.write(x, starts)

    def decode(self, x):
        """One token a request: its attention over its top_k positions, [B, H, D]."""
        self.lens += 1
        q8, weights = idx.index_prepare(x @ self.w["ik"], self.index_pool, self.tables, self.lens,
                                        q=self.heads_of(x, "iq"), weights=(x @ self.w["iw"]).float(),
                                        table=self.table)
        self.write(x)
        q = idx.rotary(self.heads_of(x, "q"), self.lens - 1, self.table)
        idx.logits_fp8(q8.view(self.B, 1, self.Hi, self.D), self.index_pool, weights, self.tables,
                       self.lens, self.max_len, out=self.logits, row_ends_out=self.row_ends)
        self.thresholds.fill_(float("inf"))
        self.counters.zero_()
        idx.threshold_select(self.logits, self.row_ends, self.thresholds, self.counters, self.slots,
                             self.top_k, self.top_k - 1, self.max_len, arrivals=self.arrivals,
                             ranges=self.ranges)
        self.q = q.view(self.B, 1, self.H, self.D)
        return self.attend(self.slots, self.ranges)

    def attend(self, slots=None, ranges=None):
        """The last step's queries over the selected positions, or over all of them."""
        return idx.attention_fp8(self.q, self.k_pool, self.v_pool, self.k_scales, self.v_scales,
                                 self.tables, self.lens, candidates=slots, ranges=ranges)[:, 0]


def run(batch=8, prompt=6000, steps=32, top_k=2048, **sizes):
    """Serves prompts of unequal lengths and `steps` decode steps from a graph; returns the layer, the
    last output and the time of a step in microseconds."""
    layer = SparseLayer(batch, prompt + steps + 8, top_k=top_k, **sizes)
    hidden = layer.w["q"].shape[0]
    g = torch.Generator("cuda").manual_seed(1)
    lens = torch.tensor([max(1, prompt - 97 * b % prompt) for b in range(batch)], dtype=torch.int32,
                        device="cuda")
    layer.prompt(torch.randn(int(lens.sum()), hidden, generator=g, device="cuda").bfloat16(), lens)
    x = torch.randn(batch, hidden, generator=g, device="cuda").bfloat16()
    layer.decode(x)  # (loads the kernels, which a capture could not)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.decode(x)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(steps):
        x.copy_(torch.randn(batch, hidden, generator=g, device="cuda"))
        graph.replay()
    torch.cuda.synchronize()
    return layer, out, (time.perf_counter() - begin) / steps * 1e6


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=6000)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=2048)
    a = ap.parse_args()
    layer, out, us = run(a.batch, a.prompt, a.steps, a.top_k)
    everything = layer.attend()
    print(f"{a.batch} requests, {layer.lens.tolist()} positions, top_k {a.top_k}: {us:.0f} us a step")
    far = ((out - everything).float().norm() / everything.float().norm()).item()
    print(f"selected against every position: {far:.3f} of the output's norm apart")
    assert idx.device_status(clear=True) == 0
    if a.top_k >= int(layer.lens.max()):
        assert far < 0.01, "the selection was everything"


if __name__ == "__main__":
    main()

"""A decoder layer's attention served with quantised weights and an 8-bit cache.

    python examples/cached_attention.py [--prompt 2048] [--steps 64] [--batch 4]

The q, k, v and o projections are block-wise mixed-precision weights; keys and values go
through the 8-bit cache.  A prompt is taken in (one grouped product, one cache write, one
attention call), then tokens are decoded one at a time from one captured HIP graph:
    q, k, v = x . Wq^T, x . Wk^T, x . Wv^T      msq.gemm_group, fp32
    cache  += k, v                               msq.kv_write
    a       = attention(q, cache)                msq.kv_attention, bf16
    y       = a . Wo^T                           msq.gemm, fp32
Weights and inputs are random; a model would encode positions in q and k between the first
two steps.  The sizes are those of a 4096-wide layer with 32 query and 8 key/value heads.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import block_wise_mixed_amd as msq  # noqa: E402
from block_wise_mixed_amd import synth  # noqa: E402


class CachedAttention:
    """Projections, cache and block table of one layer for a fixed set of sequences."""

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, batch: int,
                 max_tokens: int, block_tokens: int = 64, seed: int = 0):
        self.q_heads, self.kv_heads, self.head_dim, self.batch = q_heads, kv_heads, head_dim, batch

        def packed(rows, cols, n):
            c = synth.random_case(rows, cols, seed + n, dist={2: .3, 3: .45, 4: .2, 8: .05})
            return msq.quantize_pack(c.W, c.bits, c.perm_row, c.perm_col)

        self.qkv = [packed(q_heads * head_dim, hidden, 0), packed(kv_heads * head_dim, hidden, 1),
                    packed(kv_heads * head_dim, hidden, 2)]
        self.o = packed(hidden, q_heads * head_dim, 3)
        width = -(-max_tokens // block_tokens)
        self.max_tokens = max_tokens
        self.cache = msq.allocate_kv_cache(batch * width, kv_heads, head_dim, block_tokens)
        ids = np.random.default_rng(seed).permutation(batch * width).reshape(batch, width)
        self.table = torch.from_numpy(ids.astype(np.int32)).cuda()
        self.length = torch.zeros(batch, dtype=torch.int32, device="cuda")
        need = msq.kv_attention_workspace_bytes(self.cache, batch, q_heads, batch, 1, max_tokens)
        self.workspace = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")

    def __call__(self, x, offset=None, max_count: int = 0, workspace=None):
        """x bf16 [rows][hidden], the new tokens of all sequences (offset: ragged rows); returns
        (y fp32 [rows][hidden], q, a).  The caller's lengths grow by the rows of each sequence."""
        q, k, v = msq.gemm_group([x, x, x], self.qkv)
        heads = lambda t, h: t.view(-1, h, self.head_dim)
        q, k, v = heads(q, self.q_heads), heads(k, self.kv_heads), heads(v, self.kv_heads)
        msq.kv_write(self.cache, k, v, self.table, self.length, offset, max_count)
        if offset is None:
            self.length += x.shape[0] // self.batch
        else:
            self.length += offset[1:] - offset[:-1]
        a = msq.kv_attention(q, self.cache, self.table, self.length, offset, max_count,
                             workspace=workspace)
        return msq.gemm(a.view(x.shape[0], -1), self.o), q, a

    def decode_graph(self, x):
        """A graph of one decode step on x (bf16 [batch][hidden], a buffer the caller refills)."""
        before = self.length.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self(x, workspace=self.workspace)
            self.length.copy_(before)  # the step again, captured this time
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, _, _ = self(x, workspace=self.workspace)
        return graph, y


def run(hidden=4096, q_heads=32, kv_heads=8, head_dim=128, batch=4, prompt=2048, steps=64, seed=0):
    layer = CachedAttention(hidden, q_heads, kv_heads, head_dim, batch, prompt + steps, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda rows: torch.randn(rows, hidden, generator=gen, device="cuda").bfloat16()
    counts = [max(1, prompt - 37 * b) for b in range(batch)]  # prompts of different lengths
    offset = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    layer(new(sum(counts)), offset, max(counts))
    x = new(batch)
    graph, y = layer.decode_graph(x)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return layer, y, start.elapsed_time(end) / max(steps, 1)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--prompt", type=int, default=2048)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--batch", type=int, default=4)
    a = p.parse_args()
    layer, _, ms = run(prompt=a.prompt, steps=a.steps, batch=a.batch)
    cached = int(layer.length.sum())
    bf16 = cached * 2 * layer.kv_heads * layer.head_dim * 2
    print(f"{a.batch} sequences, {cached} tokens cached: {layer.cache.nbytes / 1e6:.1f} MB of cache "
          f"({bf16 / 1e6:.1f} MB of tokens in bf16), {1e3 * ms:.1f} us a decode step")


if __name__ == "__main__":
    main()

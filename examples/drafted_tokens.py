"""A decoder layer and head that check trees of drafted tokens, with quantised weights and an 8-bit cache.

    python examples/drafted_tokens.py [--batch 4] [--nodes 26] [--steps 32]

One step, captured in a HIP graph; lengths, trees and decisions stay on the device:
    q, k, v = x . Wq^T, x . Wk^T, x . Wv^T        msq.gemm_group, a row for every node of the trees
    sets, positions of the nodes                   msq.draft_tree
    cache += k, v; k and q rotated                 msq.kv_append
    a = attention(q, cache) by the sets            msq.kv_attention(tree=)
    logits = (a . Wo^T) . Whead^T                  msq.gemm, twice
    which nodes stay, and the next token           msq.verify_draft, by the largest logits
    those nodes' k, v one after another            msq.kv_append(source=, count=)
Weights, inputs and drafts are random, so few drafts stay; a model would draft with a smaller one.
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


class DraftedLayer:
    """Projections, head, cache and the buffers of a step for `batch` trees of `nodes` nodes."""

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, vocab: int, batch: int, nodes: int,
                 max_tokens: int, block_tokens: int = 64, seed: int = 0):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.batch, self.nodes = batch, nodes

        def packed(rows, cols, n):
            c = synth.random_case(rows, cols, seed + n, dist={2: .3, 3: .45, 4: .2, 8: .05})
            return msq.quantize_pack(c.W, c.bits, c.perm_row, c.perm_col)

        self.qkv = [packed(q_heads * head_dim, hidden, 0), packed(kv_heads * head_dim, hidden, 1),
                    packed(kv_heads * head_dim, hidden, 2)]
        self.o, self.head = packed(hidden, q_heads * head_dim, 3), packed(vocab, hidden, 4)
        width = -(-(max_tokens + nodes) // block_tokens)
        self.cache = msq.allocate_kv_cache(batch * width, kv_heads, head_dim, block_tokens)
        ids = np.random.default_rng(seed).permutation(batch * width).reshape(batch, width)
        self.table = torch.from_numpy(ids.astype(np.int32)).cuda()
        self.rot = msq.Rotary(msq.rotary_frequencies(head_dim))
        ints = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
        rows = batch * nodes
        self.length, self.parents, self.tokens = ints(batch), ints(rows) - 1, ints(rows)
        self.offset = torch.arange(0, rows + 1, nodes, dtype=torch.int32, device="cuda")
        self.x = torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda")
        need = msq.kv_attention_workspace_bytes(self.cache, rows, q_heads, batch, nodes, max_tokens + nodes)
        self.attention_space = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        need = msq.verify_draft_workspace_bytes(rows, batch, vocab, nodes, greedy=True)
        self.verify_space = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")

    def step(self):
        """One step on x, parents and tokens (buffers that the caller refills); returns (logits, token, taken,
        path) and lets the lengths grow by what was taken."""
        heads = lambda t, n: t.view(-1, n, self.head_dim)
        q, k, v = msq.gemm_group([self.x] * 3, self.qkv)
        q, k, v = heads(q, self.q_heads), heads(k, self.kv_heads), heads(v, self.kv_heads)
        at = dict(offset=self.offset, max_count=self.nodes)
        sets, positions = msq.draft_tree(self.parents, first=self.length, **at)
        q = msq.kv_append(self.cache, k, v, self.table, self.length, self.rot, q=q, positions=positions, **at)
        a = msq.kv_attention(q, self.cache, self.table, self.length + self.nodes, tree=sets,
                             workspace=self.attention_space, **at)
        y = msq.gemm(a.view(self.x.shape[0], -1), self.o).bfloat16()
        logits = msq.gemm(y, self.head)
        token, taken, path = msq.verify_draft(self.tokens, logits, parents=self.parents,
                                              workspace=self.verify_space, **at)
        msq.kv_append(self.cache, k, v, self.table, self.length, self.rot, source=path, count=taken, **at)
        self.length += taken
        return logits, token, taken, path

    def graph(self):
        """The step, captured."""
        before = self.length.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
            self.length.copy_(before)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = self.step()
        return graph, out


def run(hidden=4096, q_heads=32, kv_heads=8, head_dim=128, vocab=32000, batch=4, nodes=26, steps=32, seed=0):
    layer = DraftedLayer(hidden, q_heads, kv_heads, head_dim, vocab, batch, nodes, 1024 + steps * nodes, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    up = [int(np.random.default_rng(i).random() ** 1.5 * i) for i in range(1, nodes)]
    layer.parents.copy_(torch.tensor(([-1] + up) * batch, dtype=torch.int32))
    layer.tokens.random_(0, vocab, generator=gen)
    layer.x.normal_(generator=gen)
    graph, out = layer.graph()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return layer, out, start.elapsed_time(end) / max(steps, 1)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--nodes", type=int, default=26)
    p.add_argument("--steps", type=int, default=32)
    a = p.parse_args()
    layer, _, ms = run(batch=a.batch, nodes=a.nodes, steps=a.steps)
    print(f"{a.batch} trees of {a.nodes}: {1e3 * ms:.1f} us a step, {int(layer.length.sum())} tokens kept in {a.steps} steps")


if __name__ == "__main__":
    main()

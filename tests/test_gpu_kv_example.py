"""The cached-attention example: projections, cache write, attention and o projection together,
eager prompt and steps, and the captured decode step against eager ones."""
import os
import sys

import numpy as np
import pytest

from oracle import msq_kv as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def make(seed=1):
    import cached_attention as ex
    return ex, ex.CachedAttention(512, 8, 2, 64, 3, 200, block_tokens=32, seed=seed)


def check(msq, layer, q, a, b, rows):
    """a (bf16) against fp64 attention over the cache's own values: the kernel's bound for fp32
    queries and bf16 outputs (weights and queries rounded to f16, half a unit of bf16)."""
    L, n, D = int(layer.length[b]), rows.stop - rows.start, layer.head_dim
    k, v = msq.kv_read(layer.cache, layer.table[b:b + 1], torch.zeros(1, dtype=torch.int32, device="cuda"),
                       total=L, dtype=torch.float32)
    q, a = q[rows].cpu().numpy(), a[rows].float().cpu().numpy()
    want, _, absum, size, _ = O.attention(q, k.cpu().numpy(), v.cpu().numpy(), O.sees(L, n), 1 / np.sqrt(D))
    e = size * (2.0 ** -11 + (D + 32) * 2.0 ** -24) + 2.0 ** -20
    bound = absum * (2 * e + 2.0 ** -11 + 2.0 ** -18 + (L + 64) * 2.0 ** -24)[..., None] \
        + np.abs(want) * 2.0 ** -8 + L * 2.0 ** -31 * np.abs(v.cpu().numpy()).max()
    assert (np.abs(a - want) <= bound).all()


def test_prompt_and_steps():
    import block_wise_mixed_amd as msq
    _, layer = make()
    counts = [40, 1, 77]
    offset = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    y, q, a = layer(torch.randn(118, 512, device="cuda").bfloat16(), offset, 77)
    torch.cuda.synchronize()
    assert y.shape == (118, 512) and layer.length.tolist() == counts
    for b in range(3):
        check(msq, layer, q, a, b, slice(int(offset[b]), int(offset[b + 1])))
    for _ in range(4):
        y, q, a = layer(torch.randn(3, 512, device="cuda").bfloat16(), workspace=layer.workspace)
        torch.cuda.synchronize()
        for b in range(3):
            check(msq, layer, q, a, b, slice(b, b + 1))
    assert layer.length.tolist() == [c + 4 for c in counts]


def test_captured_steps_equal_eager_ones():
    _, one = make(seed=2)
    _, two = make(seed=2)
    prompt = torch.randn(30, 512, device="cuda").bfloat16()
    one(prompt), two(prompt)
    x = torch.randn(3, 512, device="cuda").bfloat16()
    graph, y = one.decode_graph(x)
    two(x)                       # the step that decode_graph ran before the capture
    two.length -= 1
    torch.cuda.synchronize()
    for _ in range(6):
        x.copy_(torch.randn(3, 512, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        want, _, _ = two(x)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(one.length, two.length)


def test_runs_whole():
    ex, _ = make()
    layer, y, ms = ex.run(hidden=512, q_heads=8, kv_heads=2, head_dim=128, batch=2, prompt=100, steps=5)
    assert torch.isfinite(y).all() and ms > 0
    assert layer.length.tolist() == [105, 68]

"""The drafted-tokens example: eager steps against the oracle's decisions on the same logits, and the captured
step against an eager one."""
import os
import sys

import numpy as np
import pytest

from oracle import msq_draft as T

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def make(seed=1):
    import drafted_tokens as ex
    return ex, ex.DraftedLayer(512, 8, 2, 64, 1024, 3, 9, 200, block_tokens=32, seed=seed)


def fill(layer, rng, tops=None):
    up = [[-1] + [int(rng.random() ** 1.5 * i) for i in range(1, layer.nodes)] for _ in range(layer.batch)]
    layer.parents.copy_(torch.tensor(np.array(up).ravel(), dtype=torch.int32))
    layer.tokens.copy_(torch.tensor(rng.integers(0, 1024, size=layer.tokens.numel()), dtype=torch.int32))
    layer.x.copy_(torch.from_numpy(rng.normal(size=layer.x.shape).astype(np.float32)))


def test_steps_decide_as_the_oracle():
    _, layer = make()
    rng = np.random.default_rng(0)
    kept = 0
    for _ in range(6):
        fill(layer, rng)
        before = layer.length.clone()
        cache = [t.clone() for t in (layer.cache.k_codes, layer.cache.v_codes, layer.cache.k_scale, layer.cache.v_scale)]
        logits, _, _, _ = layer.step()
        # drafts that stay: the largest logits after the rows above them, which do not hang on the drafts
        best = logits.argmax(-1).to(torch.int32).view(layer.batch, -1)
        up = layer.parents.view(layer.batch, -1)
        layer.tokens.copy_(best.gather(1, up.clamp(min=0).long()).view(-1))
        layer.tokens[::4] = 0
        layer.length.copy_(before)
        for t, was in zip((layer.cache.k_codes, layer.cache.v_codes, layer.cache.k_scale, layer.cache.v_scale), cache):
            t.copy_(was)
        logits, token, taken, path = layer.step()
        torch.cuda.synchronize()
        x, par, tok = logits.cpu().numpy(), layer.parents.view(layer.batch, -1).cpu().numpy(), layer.tokens.cpu().numpy()
        for b in range(layer.batch):
            sl = slice(b * layer.nodes, (b + 1) * layer.nodes)
            want, rows = T.verify(tok[sl], par[b], x[sl])
            assert (int(token[b]), int(taken[b])) == (want, len(rows))
            assert path[sl].tolist() == [b * layer.nodes + r for r in rows] + [-1] * (layer.nodes - len(rows))
        assert torch.equal(layer.length, before + taken)
        kept += int(taken.sum()) - layer.batch
    assert kept > 0


def test_captured_steps_equal_eager_ones():
    _, one = make(seed=2)
    _, two = make(seed=2)
    rng = np.random.default_rng(3)
    fill(one, rng)
    graph, out = one.graph()
    for _ in range(5):
        fill(one, rng)
        for name in ("x", "parents", "tokens"):
            getattr(two, name).copy_(getattr(one, name))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = two.step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(one.length, two.length)


def test_runs_whole():
    ex, _ = make()
    layer, out, ms = ex.run(hidden=512, q_heads=8, kv_heads=2, head_dim=128, vocab=1024, batch=2, nodes=5, steps=4)
    assert torch.isfinite(out[0]).all() and ms > 0
    assert all(4 <= n <= 20 for n in layer.length.tolist())

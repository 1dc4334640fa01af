"""The operators on drafted tokens together, as a program has them: the sets of a tree, rotated append, attention
by the sets, verification, and the drafts that stay appended over the others, all lengths on the device; eager and
as one captured graph replayed with new inputs.  Against the oracles: cache and decisions bit for bit, attention
within the bounds of test_gpu_kv.py."""
import numpy as np
import pytest

from oracle import msq_draft as T
from oracle import msq_kv as O
from oracle import msq_rotary as R
from test_gpu_kv import Pair, i32, msq, offsets, rounded  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Step:
    """One layer and the decision on its drafts for sequences of a fixed number of rows."""

    def __init__(self, msq, counts, H, G, D, P, V, way, dtype, interleaved, seed):
        self.msq, self.counts, self.G, self.V, self.way, self.dtype = msq, counts, G, V, way, dtype
        self.interleaved = interleaved
        B, n = len(counts), sum(counts)
        width = -(-300 // P)
        self.table = np.random.default_rng(seed).permutation(B * width).reshape(B, width)
        self.p = Pair(msq, B * width, H, D, P, seed=seed, fill=3.0)
        self.rng = self.p.rng
        self.rot = msq.Rotary(msq.rotary_frequencies(D, factor=4.0, original=64), interleaved, 1.1)
        self.length = i32([0] * B)
        self.off = offsets(counts)
        self.dev = dict(offset=i32(self.off), table=i32(self.table), counts=i32(counts), parents=i32([-1] * n),
                        tokens=i32([0] * n), k=torch.zeros(n, H, D, dtype=dtype, device="cuda"),
                        v=torch.zeros(n, H, D, dtype=dtype, device="cuda"),
                        q=torch.zeros(n, H * G, D, dtype=dtype, device="cuda"),
                        target=torch.zeros(n, V, device="cuda"), draft=torch.zeros(n, V, device="cuda"),
                        uniform=torch.zeros(n, device="cuda"))
        need = msq.kv_attention_workspace_bytes(self.p.gpu, n, H * G, B, max(counts), width * P)
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        need = msq.verify_draft_workspace_bytes(n, B, V, max(counts), greedy=way == "largest")
        self.ws2 = torch.empty(need, dtype=torch.uint8, device="cuda")

    def new_inputs(self):
        rng, n, d = self.rng, sum(self.counts), self.dev
        self.host = h = {}
        for name in "kvq":
            h[name], t = rounded(rng.normal(size=d[name].shape) * np.exp(rng.normal() * 0.5), self.dtype)
            d[name].copy_(t)
        h["parents"] = [np.array([-1] + [int(rng.random() ** 1.5 * i) for i in range(1, c)])[:c] for c in self.counts]
        d["parents"].copy_(i32(np.concatenate(h["parents"])))
        x = rng.normal(size=(n, self.V)) * 2
        for name, y in (("target", x), ("draft", x + rng.normal(size=x.shape) * 0.5)):
            e = np.exp(y - y.max(1, keepdims=True))
            h[name] = (e / e.sum(1, keepdims=True)).astype(np.float32)
            d[name].copy_(torch.from_numpy(h[name]))
        tokens = []
        for b, c in enumerate(self.counts):
            for i in range(c):
                row = h["draft"][self.off[b] + max(h["parents"][b][i], 0)].astype(float)
                tokens.append(int(row.argmax()) if self.way == "largest" else int(rng.choice(self.V, p=row / row.sum())))
        h["tokens"] = np.array(tokens)
        h["uniform"] = rng.random(n).astype(np.float32)
        d["tokens"].copy_(i32(tokens))
        d["uniform"].copy_(torch.from_numpy(h["uniform"]))

    def run(self):
        msq, d, most = self.msq, self.dev, max(self.counts)
        sets, at = msq.draft_tree(d["parents"], d["offset"], self.length, max_count=most)
        q = msq.kv_append(self.p.gpu, d["k"], d["v"], d["table"], self.length, self.rot, q=d["q"], positions=at,
                          offset=d["offset"], max_count=most)
        a = msq.kv_attention(q, self.p.gpu, d["table"], self.length + d["counts"], d["offset"], max_count=most,
                             out_dtype=torch.float32, workspace=self.ws, tree=sets)
        token, taken, path = msq.verify_draft(
            d["tokens"], d["target"], d["offset"], parents=d["parents"], draft=d["draft"] if self.way == "drawn" else None,
            uniform=None if self.way == "largest" else d["uniform"], max_count=most, workspace=self.ws2)
        msq.kv_append(self.p.gpu, d["k"], d["v"], d["table"], self.length, self.rot, offset=d["offset"],
                      max_count=most, source=path, count=taken)
        self.length += taken
        return q, a, token, taken, path

    def check(self, before, q, a, token, taken, path):
        torch.cuda.synchronize()
        h, ref, D = self.host, self.p.ref, self.p.D
        f = self.rot.frequencies.cpu().numpy()
        first = [int(b) for b in before]
        sets = [T.ancestors(p) for p in h["parents"]]
        at = np.concatenate([s.sum(1) - 1 + b for s, b in zip(sets, first)])
        turn = lambda x, at: R.rotate(x, at, f, self.interleaved, 1.1)
        q_ref = torch.from_numpy(turn(h["q"], at)).to(self.dtype)
        assert torch.equal(q.cpu(), q_ref)
        ref.write(turn(h["k"], at), h["v"], self.table, first, self.off)
        for b, n in enumerate(self.counts):
            sl, L = slice(self.off[b], self.off[b] + n), first[b] + n
            step = ref.scale["v"][self.table[b][np.arange(L) // ref.P]]
            want, _, absum, size, big = O.attention(q_ref[sl].float().numpy(), ref.values("k", self.table[b], 0, L),
                                                    ref.values("v", self.table[b], 0, L), T.tree_sees(L, sets[b]),
                                                    1 / np.sqrt(D), step)
            e = size * (2.0 ** -22 + (D + 32) * 2.0 ** -24) + 2.0 ** -20
            bound = absum * (2 * e + 2.0 ** -22 + 2.0 ** -18 + (L + 64) * 2.0 ** -24)[..., None] \
                + (L * 2.0 ** -31 * 127 * big)[..., None]
            assert (np.abs(a[sl].cpu().numpy() - want) <= bound).all(), b
            t, rows = T.verify(h["tokens"][sl], h["parents"][b], h["target"][sl].astype(float),
                               h["draft"][sl].astype(float) if self.way == "drawn" else None,
                               None if self.way == "largest" else h["uniform"][sl])
            assert (int(token[b]), int(taken[b])) == (t, len(rows)), b
            assert path[sl].tolist() == [self.off[b] + r for r in rows] + [-1] * (n - len(rows)), b
            rows = np.array(rows) + self.off[b]
            ref.write(turn(h["k"][rows], np.arange(len(rows)) + first[b]), h["v"][rows], self.table[b:b + 1],
                      [first[b]], [0, len(rows)])
        self.p.check()
        assert self.length.tolist() == [x + int(y) for x, y in zip(first, taken)]


@pytest.mark.parametrize("way,dtype,D,P,interleaved", [
    ("drawn", torch.bfloat16, 128, 64, False), ("chosen", torch.float32, 64, 32, True),
    ("largest", torch.bfloat16, 256, 32, False), ("drawn", torch.float32, 64, 128, True)])
def test_steps_eager_and_captured(msq, way, dtype, D, P, interleaved):
    print("step", way, dtype, D, P, flush=True)
    s = Step(msq, [26, 1, 9, 33], 2, 3, D, P, 501, way, dtype, interleaved, seed=D + P)
    for _ in range(2):
        s.new_inputs()
        before = s.length.clone()
        s.check(before, *s.run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.run()
    for _ in range(4):
        s.new_inputs()
        before = s.length.clone()
        torch.cuda.synchronize()
        graph.replay()
        s.check(before, *out)

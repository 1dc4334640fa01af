"""Rotary positions and drafted tokens at the limits of their sizes: addresses past 32 bits, rows that are left
alone, calls side by side on several streams, the most rows and entries."""
import numpy as np
import pytest

from oracle import msq_draft as T
from test_gpu_kv import i32, msq  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_rotary_addresses_past_32_bits(msq):
    """Rows 2^31 + 64 values apart, and heads 2^31 apart, in and out."""
    f = msq.rotary_frequencies(64)
    rot = msq.Rotary(f)
    far = 2 ** 31 + 64
    for dtype in (torch.bfloat16, torch.float32):
        base = torch.empty(far + 1024, dtype=dtype, device="cuda")
        for shape, stride in (((2, 3, 64), (far, 64, 1)), ((3, 2, 64), (64, far, 1))):
            x = base.as_strided(shape, stride)
            near = torch.randn(shape, device="cuda").to(dtype)
            x.copy_(near)
            at = i32([5, 100000, 7][:shape[0]])
            want = msq.rotary(near, at, rot)
            assert torch.equal(msq.rotary(x, at, rot), want)
            assert msq.rotary(x, at, rot, out=x) is x and torch.equal(x.contiguous(), want)
        del base


def test_append_into_a_large_cache(msq):
    """Blocks past 4 GB of codes; the append's reads and writes against those of a small cache."""
    H, D, P = 8, 256, 256
    blocks = 8400  # x 512 KB: 4.4 GB for keys, as much for values
    big = msq.allocate_kv_cache(blocks, H, D, P)
    small = msq.allocate_kv_cache(4, H, D, P)
    rot = msq.Rotary(msq.rotary_frequencies(D))
    k, v = (torch.randn(600, H, D, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(600, 16, D, device="cuda").bfloat16()
    ids = {id(big): i32([[8399, 8250, 8193]]), id(small): i32([[0, 2, 1]])}
    for n, at in ((600, 0), (1, 600), (26, 601)):
        got = [msq.kv_append(c, k[:n], v[:n], ids[id(c)], i32([at]), rot, q=q[:n]) for c in (big, small)]
        assert torch.equal(*got)
    for a, b in zip(*(msq.kv_read(c, ids[id(c)], i32([0]), total=627, dtype=torch.float32) for c in (big, small))):
        assert torch.equal(a, b)
    sets, _ = msq.draft_tree(i32(list(range(-1, 25))))
    out = [msq.kv_attention(q[:26], c, ids[id(c)], i32([627]), tree=sets, out_dtype=torch.float32) for c in (big, small)]
    assert torch.equal(*out)


def test_verify_addresses_past_32_bits(msq):
    """2100 rows of 2^20 entries, 2^31 of them passed; the last sequence's rows lie behind."""
    V, n = 1 << 20, 2100
    target = torch.zeros(n, V, dtype=torch.bfloat16, device="cuda")
    tokens = torch.randint(0, V, (n,), dtype=torch.int32, device="cuda")
    rows = torch.arange(n, device="cuda")
    target[rows, (rows * 977 + 13) % V] = 0.5
    target[rows, (rows * 31 + 1000000) % V] = 0.375
    offset = i32([0, 700, 1400, 2090, 2100])
    tokens[1:] = ((rows[:-1] * 977 + 13) % V).to(torch.int32)   # the larger of the row before
    tokens[2097] = 5                                             # but here
    u = torch.full((n,), 0.3, device="cuda")
    for uniform in (None, u):
        token, taken, path = msq.verify_draft(tokens, target, offset, uniform=uniform, max_count=700)
        assert taken.tolist() == [700, 700, 690, 7]
        last = [699, 1399, 2089, 2096]
        assert token.tolist() == [(r * 977 + 13) % V if uniform is None else
                                  [(r * 977 + 13) % V, (r * 31 + 1000000) % V][int(
                                      (0.3 * 0.875 > 0.5) if (r * 977 + 13) % V < (r * 31 + 1000000) % V else
                                      (0.3 * 0.875 <= 0.375))] for r in last]
        assert path[2090:2097].tolist() == list(range(2090, 2097)) and (path[2097:] == -1).all()


def test_verify_many_entries(msq):
    """A vocabulary past 2^24: slices of more than 1024 entries, indexes that fp32 does not hold."""
    V = (1 << 24) + 12345
    p = torch.zeros(2, V, device="cuda")
    at = torch.tensor([3, 1 << 23, (1 << 24) + 1, V - 2, V - 1], device="cuda")
    p[:, at] = torch.tensor([.1, .2, .3, .2, .2], device="cuda")
    for u, want in ((0.05, 3), (0.25, 1 << 23), (0.45, (1 << 24) + 1), (0.7, V - 2), (0.9, V - 1), (1.0, V - 1)):
        token, taken, _ = msq.verify_draft(i32([0, 7]), p, uniform=torch.tensor([u, 0.5], device="cuda"))
        assert (token.tolist(), taken.tolist()) == ([want], [1])
    q = torch.zeros_like(p)
    q[:, at[2]] = 1.0                       # all of it drawn there: .3 of 1 is kept, the rest is the others'
    for u0, u1, want in ((0.2, 0.29, (1, 2)), (0.2, 0.31, (1 << 23, 1)), (0.6, 0.31, (V - 2, 1)), (0.99, 0.31, (V - 1, 1))):
        token, taken, _ = msq.verify_draft(i32([0, (1 << 24) + 1]), p, draft=q, uniform=torch.tensor([u0, u1], device="cuda"))
        if want[1] == 1:
            assert (token.tolist(), taken.tolist()) == ([want[0]], [1])
        else:
            assert taken.tolist() == [2]
    token, _, _ = msq.verify_draft(i32([0, 7]), p)
    assert token.tolist() == [(1 << 24) + 1]


@pytest.mark.parametrize("greedy", [False, True])
def test_verify_leaves_other_rows(msq, greedy):
    """path outside every sequence, and outputs of empty sequences."""
    rng = np.random.default_rng(0)
    n, V = 12, 50
    p = torch.from_numpy(rng.random((n, V)).astype(np.float32)).cuda()
    path = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    token, taken = (torch.full((4,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    tokens, offset, u = i32([1] * n), i32([2, 5, 5, 9, 9]), torch.full((n,), 0.5, device="cuda")
    d = msq._Draft()
    ws = torch.empty(msq.verify_draft_workspace_bytes(n, 4, V, 4, greedy), dtype=torch.uint8, device="cuda")
    msq._DRAFT.pack_into(d, 0, 4, offset.data_ptr(), n, 4, V, tokens.data_ptr(), 0, p.data_ptr(), V, 0, V, 1,
                         0 if greedy else u.data_ptr(), token.data_ptr(), taken.data_ptr(), path.data_ptr())
    assert msq.load_library().msq_verify_draft(d, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert (path[:2] == 77).all() and (path[9:] == 77).all() and not (path[2:9] == 77).any()
    assert token.tolist()[1::2] == [-1, -1] and taken.tolist()[1::2] == [0, 0]


def test_calls_side_by_side(msq):
    """The same calls on three streams at once, each with its own inputs and workspaces, against one after
    another."""
    rng = np.random.default_rng(2)
    H, G, D, P, V, n = 2, 4, 128, 64, 20000, 26
    jobs = []
    for s in range(3):
        B = s + 1
        table = i32(rng.permutation(B * 40).reshape(B, 40))
        up = np.concatenate([[-1] + [int(rng.random() ** 1.5 * i) for i in range(1, n)] for _ in range(B)])
        x = torch.randn(B * n, V, device="cuda")
        job = dict(cache=msq.allocate_kv_cache(B * 40, H, D, P), table=table, first=i32([2000 - 100 * s] * B),
                   k=torch.randn(B * n, H, D, device="cuda"), v=torch.randn(B * n, H, D, device="cuda"),
                   q=torch.randn(B * n, H * G, D, device="cuda"), parents=i32(up), offset=i32(np.arange(B + 1) * n),
                   tokens=x.topk(1, -1).indices[:, 0].to(torch.int32), target=torch.softmax(x, -1),
                   draft=torch.softmax(x + 0.5 * torch.randn_like(x), -1), u=torch.rand(B * n, device="cuda"))
        fill = torch.randn(B * 2000, H, D, device="cuda")
        msq.kv_write(job["cache"], fill, fill, table, i32([0] * B))
        jobs.append(job)
    rot = msq.Rotary(msq.rotary_frequencies(D))

    def run(j, **kw):
        sets, at = msq.draft_tree(j["parents"], j["offset"], j["first"], max_count=n, **kw)
        q = msq.kv_append(j["cache"], j["k"], j["v"], j["table"], j["first"], rot, q=j["q"], positions=at,
                          offset=j["offset"], max_count=n, **kw)
        a = msq.kv_attention(q, j["cache"], j["table"], j["first"] + n, j["offset"], max_count=n, tree=sets,
                             out_dtype=torch.float32, **kw)
        one = msq.verify_draft(j["tokens"], j["target"], j["offset"], parents=j["parents"], uniform=j["u"],
                               draft=j["draft"], max_count=n, **kw)
        two = msq.verify_draft(j["tokens"], j["target"], j["offset"], parents=j["parents"], max_count=n, **kw)
        return [sets, at, q, a, *one, *two]

    for j in jobs:
        run(j)  # (the scales have grown now)
    want = [run(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        got = []
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(run(j))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_largest_trees_together(msq):
    """1024 rows a sequence, as many as a call takes: sets, attention (against the causal mask for chains) and
    verification."""
    H, D, P, n = 1, 64, 64, 1024
    cache = msq.allocate_kv_cache(40, H, D, P)
    table = i32(np.random.default_rng(3).permutation(40).reshape(2, 20))
    k, v = (torch.randn(2 * 1200, H, D, device="cuda").bfloat16() for _ in range(2))
    msq.kv_write(cache, k, v, table, i32([0, 0]))
    q = torch.randn(2 * n, 2, D, device="cuda").bfloat16()
    chain = i32(list(range(-1, n - 1)) * 2)
    sets, at = msq.draft_tree(chain, first=i32([176, 176]), batch=2)
    assert sets.shape == (2 * n, 32) and at[:n].tolist() == list(range(176, 1200))
    a = msq.kv_attention(q, cache, table, i32([1200, 1200]), tree=sets)
    b = msq.kv_attention(q, cache, table, i32([1200, 1200]))
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()
    rng = np.random.default_rng(4)
    tokens = rng.integers(0, 40, size=n)
    up = np.array([-1] + [int(rng.random() * i) for i in range(1, n)])
    p = rng.random((n, 40)).astype(np.float32)
    p /= p.sum(1, keepdims=True)
    u = rng.random(n).astype(np.float32) * 0.1
    for kw in (dict(uniform=torch.from_numpy(u).cuda()), dict(uniform=torch.from_numpy(u).cuda(), draft=torch.from_numpy(p).cuda()), {}):
        token, taken, path = msq.verify_draft(i32(tokens), torch.from_numpy(p).cuda(), parents=i32(up), **kw)
        want, rows = T.verify(tokens, up, p.astype(float), p.astype(float) if "draft" in kw else None, u if kw else None)
        assert (int(token), int(taken), path[:len(rows)].tolist()) == (want, len(rows), rows)

"""Sets of draft trees, and attention by such sets over the 8-bit cache, against the oracles.  Error
bounds as in test_gpu_kv.py; for fp32 results queries and weights count by 22 bits, so that 2^-11 there is 2^-22
here (a weight's second term ends at 2^-25, which the term for small weights has already)."""
import numpy as np
import pytest

from oracle import msq_draft as T
from oracle import msq_kv as O
from test_gpu_kv import Pair, i32, msq, offsets, rounded, scattered  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def random_tree(rng, n):
    return np.array([-1] + [int(rng.random() ** 1.5 * i) for i in range(1, n)])[:n]


def as_words(sets, width):
    """int32 [rows][width] of the sequences' bool sets."""
    return torch.from_numpy(np.concatenate([T.words(s, width) for s in sets]).view(np.int32)).cuda()


# ---------------------------------------------------------------- sets

@pytest.mark.parametrize("counts", [[1], [26], [5, 0, 64, 33, 1], [300, 31, 32], [1024, 700]])
def test_draft_tree(msq, counts):
    rng = np.random.default_rng(sum(counts))
    parents = [random_tree(rng, n) for n in counts]
    for p in parents:  # what is no smaller row makes a root
        if len(p) > 4:
            p[2], p[3] = 2, len(p) + 5
    first = rng.integers(0, 1 << 30, size=len(counts))
    off = offsets(counts)
    for most in (0, max(counts)):
        sets, at = msq.draft_tree(i32(np.concatenate(parents)), i32(off), i32(first), max_count=most)
        width = sets.shape[1]
        assert width == max(1, -(-min(most or sum(counts), 1024) // 32))
        want = [T.ancestors(p) for p in parents]
        assert torch.equal(sets, as_words(want, width))
        depth = np.concatenate([w.sum(1) - 1 + f for w, f in zip(want, first)])
        assert np.array_equal(at.cpu().numpy(), depth)
    assert np.array_equal(msq.draft_tree(i32(np.concatenate(parents)), i32(off))[1].cpu().numpy(),
                          np.concatenate([w.sum(1) - 1 for w in want]))


def test_draft_tree_chains_uniform_and_left_rows(msq):
    """Sequences of one length; the longest chain; rows outside every sequence."""
    sets, at = msq.draft_tree(i32(list(range(-1, 1023))))
    assert np.array_equal(at.cpu().numpy(), np.arange(1024))
    assert torch.equal(sets, as_words([np.tril(np.ones((1024, 1024), bool))], 32))
    sets, at = msq.draft_tree(i32([-1, 0, 0] * 5), batch=5)
    assert sets.cpu().tolist() == [[1], [3], [5]] * 5
    assert msq.draft_tree(i32([]), batch=0)[0].shape[0] == 0
    lib = msq.load_library()
    s, t = torch.full((8, 1), 7, dtype=torch.int32, device="cuda"), torch.full((8,), 7, dtype=torch.int32, device="cuda")
    par, off = i32([-1] * 8), i32([1, 3, 3, 6])
    assert lib.msq_draft_tree(par.data_ptr(), off.data_ptr(), 3, 8, 2, None, s.data_ptr(), 1, t.data_ptr(),
                              torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert s[:, 0].tolist() == [7, 1, 2, 1, 2, 7, 7, 7] and t.tolist() == [7, 0, 0, 0, 0, 7, 7, 7]


# ---------------------------------------------------------------- attention

def attend(msq, p, q, table, lens, sets, words=None, dtype=torch.bfloat16, out=torch.float32, window=0, **kw):
    counts = [len(s) for s in sets]
    off = offsets(counts)
    q, qt = rounded(q, dtype)
    words = words or max(1, -(-max(counts) // 32))
    to = torch.full(qt.shape, float("nan"), dtype=out, device="cuda")
    got, lse = msq.kv_attention(qt, p.gpu, i32(table), i32(lens), i32(off), max_count=max(counts), window=window,
                                out=to, return_lse=True, tree=as_words(sets, words), **kw)
    torch.cuda.synchronize()
    table = np.asarray(table)
    P, D = p.ref.P, p.D
    for b, L in enumerate(lens):
        n, sl = counts[b], slice(off[b], off[b + 1])
        if not n:
            continue
        seen = np.zeros((n, n), bool)  # rows past the words are in no set
        seen[:, :32 * words] = sets[b][:, :32 * words]
        mask = T.tree_sees(L, seen, window)
        held = min(L, table.shape[1] * P)
        here = np.zeros(held, bool)
        ids = table[b][np.arange(held) // P]
        here[:] = (ids >= 0) & (ids < p.gpu.num_blocks)
        mask = mask[:, :held] & here
        row = np.where((table[b] >= 0) & (table[b] < p.gpu.num_blocks), table[b], 0)
        step = p.ref.scale["v"][row[np.arange(held) // P]]
        want, wl, absum, size, big = O.attention(q[sl], p.ref.values("k", row, 0, held), p.ref.values("v", row, 0, held),
                                                 mask, kw.get("scale", 0) or 1 / np.sqrt(D), step)
        term = 2.0 ** -22 if out == torch.float32 else 2.0 ** -11
        r = 0.0 if dtype == torch.bfloat16 else term
        e = size * (r + (D + 32) * 2.0 ** -24) + 2.0 ** -20
        bound = absum * (2 * e + term + 2.0 ** -18 + (held + 64) * 2.0 ** -24)[..., None] \
            + (held * 2.0 ** -31 * 127 * big)[..., None] + 1e-37
        if out == torch.bfloat16:
            bound = bound + np.abs(want) * 2.0 ** -8
        g, l = got[sl].float().cpu().numpy(), lse[sl].cpu().numpy()
        assert np.isfinite(g).all()
        assert (np.abs(g - want) <= bound).all(), (b, float((np.abs(g - want) / bound).max()))
        empty = ~mask.any(1)
        assert (g[empty] == 0).all() and np.isneginf(l[empty]).all()
        lb = e + np.abs(wl, where=np.isfinite(wl), out=np.zeros_like(wl)) * 2.0 ** -22 + (held + 64) * 2.0 ** -24
        assert (np.abs(l[~empty] - wl[~empty]) <= lb[~empty]).all()
    return got


CASES = [  # D, P, H, G, cached before the call, rows: few rows and many, in one part and several
    (64, 32, 2, 3, [300, 33, 0], [5, 1, 2]), (64, 64, 1, 8, [700, 61], [26, 64]),
    (128, 64, 2, 4, [751], [26]), (128, 32, 1, 4, [3000, 100, 7], [33, 2, 40]),
    (128, 128, 1, 1, [127, 128, 129], [130, 31, 96]), (256, 64, 1, 2, [500, 63], [26, 33]),
    (256, 32, 1, 1, [9000], [4])]


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("D,P,H,G,before,counts", CASES)
def test_trees(msq, D, P, H, G, before, counts, dtype, out):
    print("tree", D, P, H, G, before, counts, dtype, flush=True)
    rng = np.random.default_rng(D + sum(counts))
    lens = [a + n for a, n in zip(before, counts)]
    table, blocks = scattered(rng, lens, P)
    p = Pair(msq, blocks, H, D, P, seed=D, fill=float("inf"))
    p.write(table, [0] * len(lens), lens)
    sets = [T.ancestors(random_tree(rng, n)) for n in counts]
    q = rng.normal(size=(sum(counts), H * G, D))
    wide = np.concatenate([table, np.full((len(lens), 400), -1)], 1)
    for t in (table, wide):
        for window in (0, 1, 3, 40, 500):
            attend(msq, p, q, t, lens, sets, dtype=dtype, out=out, window=window)


def many(msq, D, want_waves):
    """Sizes for which the kernel for many rows takes the call, found by its plan: (H, G, before, rows,
    extra idle sequences, table width)."""
    P = 64
    c = msq.allocate_kv_cache(1, 1, D, P)
    for rows, G in ((64, 8), (100, 8), (130, 8), (512, 1)):
        for idle in (0, 10, 30, 60, 100, 200, 300):
            for width in (16, 64, 256, 1024, 4096):
                if (idle + 1) * width > 4_000_000:
                    continue
                plan = msq.kv_attention_plan(c, rows, G, 1 + idle, width, rows)
                if plan["tile_rows"] == 32 * want_waves and plan["wavefronts"] == want_waves:
                    yield G, rows, idle, width, plan


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("D,waves", [(64, 4), (64, 8), (128, 4), (128, 8), (256, 4)])
def test_trees_many_rows(msq, D, waves, split):
    P = 64
    found = [f for f in many(msq, D, waves) if (f[4]["parts"] > 1) == split]
    if not found:
        pytest.skip("no plan of these sizes")
    G, n, idle, width, plan = found[0]
    print("many", D, waves, G, n, idle, width, plan, flush=True)
    rng = np.random.default_rng(D + waves)
    before = min(900, width * P - n - 3)
    lens, counts = [before + n], [n]
    table, blocks = scattered(rng, lens, P)
    p = Pair(msq, blocks, 1, D, P, seed=D, fill=float("nan"))
    p.write(table, [0], lens)
    table = np.concatenate([table, np.full((1, width - table.shape[1]), -1)], 1)
    table = np.concatenate([table, np.full((idle, width), -1)])
    q = rng.normal(size=(n, G, D))
    for sets, window in ((T.ancestors(random_tree(rng, n)), 0), (T.ancestors(random_tree(rng, n)), 2),
                         (rng.random((n, n)) < 0.2, 0), (rng.random((n, n)) < 0.5, 20)):
        counts_all = [sets] + [np.zeros((0, 0), bool)] * idle
        attend(msq, p, q, table, lens + [0] * idle, counts_all, window=window)
        attend(msq, p, q, table, lens + [0] * idle, counts_all, window=window, dtype=torch.float32)


@pytest.mark.parametrize("D,H,G,before,counts", [
    (64, 1, 4, [300, 256, 10], [9, 26, 5]), (128, 2, 4, [2500, 700], [26, 3]), (64, 2, 3, [6100, 31, 4000], [17, 0, 6]),
    (128, 1, 8, [21000, 5], [3, 4]), (64, 1, 5, [30000], [7]), (128, 8, 8, [900, 1300, 33], [33, 26, 40])])
def test_rows_on_middle_lengths(msq, D, H, G, before, counts):
    """Row tiles in one part, in parts joined inside the launch and by a launch of their own, each twice with
    a workspace that holds what the last call left."""
    P, rng = 64, np.random.default_rng(D + G)
    lens = [a + n for a, n in zip(before, counts)]
    table, blocks = scattered(rng, lens, P)
    table[0, 1] = -1
    p = Pair(msq, blocks, H, D, P, seed=G, fill=float("nan"))
    p.write(table, [0] * len(lens), lens)
    q = rng.normal(size=(sum(counts), H * G, D))
    most = max(counts)
    ws = torch.zeros(msq.kv_attention_workspace_bytes(p.gpu, sum(counts), H * G, len(lens), most, table.shape[1] * P),
                     dtype=torch.uint8, device="cuda")
    for sets, window in (([T.ancestors(random_tree(rng, n)) for n in counts], 0),
                         ([rng.random((n, n)) < 0.3 for n in counts], 600)):
        for dtype, out in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.float32)):
            once, again = (attend(msq, p, q, table, lens, sets, dtype=dtype, out=out, window=window, workspace=ws)
                           for _ in range(2))
            assert torch.equal(once, again)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("D,waves", [(64, 4), (128, 4), (128, 8), (256, 4)])
def test_last_rows_of_many(msq, D, waves, G, split):
    """Row tiles of one row, of 16, 17, 32 and 33, alone or behind full ones, in the kernel for many rows: its
    workgroups take those of up to 32 otherwise."""
    P, tile = 64, 32 * waves // G
    n = 2 * tile + 5
    counts = [n, tile + 1, tile + max(1, 16 // G), tile + 16 // G + 1, tile + 32 // G, tile + 32 // G + 1, 1, 2, 32 // G, 0]
    c = msq.allocate_kv_cache(1, 1, D, P)
    plans = [(w, i, msq.kv_attention_plan(c, sum(counts), G, len(counts) + i, w, n)) for w in (12, 20, 40, 64)
             for i in (0, 5, 20, 50, 100, 200)]
    plans = [f for f in plans if f[2]["wavefronts"] == waves and f[2]["tile_rows"] == 32 * waves
             and (f[2]["parts"] > 1) == split]
    if not plans:
        pytest.skip("no plan of these sizes")
    width, idle, plan = plans[0]
    print("last rows", D, waves, G, width, idle, plan, flush=True)
    rng = np.random.default_rng(D + waves + G)
    longest = width * P - n
    lens = [b + m for b, m in zip([longest, longest - 70, 0, 33, longest - 1, 300, 200, longest, 64, 100], counts)]
    table, blocks = scattered(rng, lens, P)
    table = np.concatenate([table, np.full((len(lens), width - table.shape[1]), -1)], 1)
    table[1, 2] = -1  # an absent block
    p = Pair(msq, blocks, 1, D, P, seed=D, fill=float("nan"))
    p.write(table, [0] * len(lens), lens)
    table = np.concatenate([table, np.full((idle, width), -1)])
    q = rng.normal(size=(sum(counts), G, D))
    rest = [np.zeros((0, 0), bool)] * idle
    for sets, window in (([T.ancestors(random_tree(rng, m)) for m in counts], 0),
                         ([rng.random((m, m)) < 0.3 for m in counts], 40)):
        for dtype, out in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.float32)):
            attend(msq, p, q, table, lens + [0] * idle, sets + rest, dtype=dtype, out=out, window=window)


@pytest.mark.parametrize("D,G", [(64, 1), (128, 16), (256, 3)])
def test_any_sets(msq, D, G):
    """Sets that are no trees: empty ones, ones without the row itself, of later rows; a cache that holds
    fewer tokens than the call has rows, none at all, or more than the table; words that do not reach."""
    P, rng = 32, np.random.default_rng(D)
    lens = [200, 20, 0, 90, 64]
    counts = [40, 40, 7, 70, 64]
    table, blocks = scattered(rng, [200] * 5, P)
    p = Pair(msq, blocks, 1, D, P, seed=D, fill=float("nan"))
    p.write(table, [0] * 5, lens)
    q = rng.normal(size=(sum(counts), G, D))
    for density in (0.0, 0.1, 0.6, 1.0):
        sets = [rng.random((n, n)) < density for n in counts]
        for window in (0, 1, 17, 60):
            attend(msq, p, q, table, lens, sets, window=window)
        attend(msq, p, q, table, lens, sets, words=1)
        attend(msq, p, q, table, lens, sets, words=5, dtype=torch.float32)
    attend(msq, p, q, table[:, :2], lens, [rng.random((n, n)) < 0.5 for n in counts], window=100)
    gone = table.copy()
    gone[:, 1] = -1
    attend(msq, p, q, gone, lens, [rng.random((n, n)) < 0.5 for n in counts])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chains_are_causal(msq, D):
    """A chain's sets give what the causal mask gives: of many rows, which are split otherwise, within the
    rounding of both to bf16; bit for bit where the plan is the same (16 rows a head)."""
    chains_are_causal(msq, D, [700, 90], [33, 20], False)
    chains_are_causal(msq, D, [700, 90], [4, 3], True)


def chains_are_causal(msq, D, lens, counts, same):
    P, rng = 64, np.random.default_rng(D)
    table, blocks = scattered(rng, lens, P)
    p = Pair(msq, blocks, 2, D, P, seed=D)
    p.write(table, [0, 0], lens)
    q = torch.randn(sum(counts), 8, D, device="cuda").bfloat16()
    off = i32(offsets(counts))
    sets, _ = msq.draft_tree(i32(np.concatenate([np.arange(n) - 1 for n in counts])), off, max_count=max(counts))
    for window in (0, 10, 300):
        # (bf16 results: fp32 ones have weights in two terms here)
        a = msq.kv_attention(q, p.gpu, i32(table), i32(lens), off, max_count=max(counts), window=window, tree=sets)
        b = msq.kv_attention(q, p.gpu, i32(table), i32(lens), off, max_count=max(counts), window=window)
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()
        if same and not window:
            assert torch.equal(a, b)


def test_rows_left_alone_streams_and_graph(msq):
    P, H, D = 64, 2, 128
    rng = np.random.default_rng(1)
    lens = [2000, 300]
    table, blocks = scattered(rng, [2100, 400], P)
    p = Pair(msq, blocks, H, D, P, seed=5)
    p.write(table, [0, 0], lens)
    t, n = i32(table), i32(lens)
    off = i32([2, 28, 50])
    q = torch.randn(55, 8, D, device="cuda").bfloat16()
    parents = i32(np.concatenate([[0, 0], random_tree(rng, 26), random_tree(rng, 22), [0] * 5]))
    out = torch.full((55, 8, D), 7.0, device="cuda")
    sets, _ = msq.draft_tree(parents, off, max_count=26)
    ws = torch.empty(max(256, msq.kv_attention_workspace_bytes(p.gpu, 55, 8, 2, 26, 2100)), dtype=torch.uint8, device="cuda")
    call = lambda **kw: msq.kv_attention(q, p.gpu, t, n, off, max_count=26, tree=sets, workspace=ws, **kw)
    call(out=out)
    assert (out[:2] == 7).all() and (out[50:] == 7).all() and not (out[2:50] == 7).all(-1).any()
    want = call(out_dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(out_dtype=torch.float32, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[2:50], want[2:50])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sets, _ = msq.draft_tree(parents, off, max_count=26)
        y = call()
    for step in range(4):
        parents[2:28] = i32(random_tree(rng, 26))
        q.copy_(torch.randn_like(q))
        n -= 5
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = sets
        sets, _ = msq.draft_tree(parents, off, max_count=26)
        assert torch.equal(kept[2:50], sets[2:50])
        assert torch.equal(y[2:50], call()[2:50]), step
        sets = kept


def planned(msq, D, shapes, want):
    """The first (counts, heads a group, idle sequences, table entries) whose call by sets has the plan (tile rows,
    wavefronts, join) that is wanted."""
    c = msq.allocate_kv_cache(1, 1, D, 64, device="cpu")
    for counts, G in shapes:
        for width in (4, 8, 16, 20, 40, 64, 256, 1024, 4096):
            for idle in (0, 4, 10, 30, 60, 75, 100, 165, 200, 255, 300):
                plan = msq.kv_attention_plan(c, sum(counts), G, len(counts) + idle, width, max(counts), tree=True)
                if (plan["tile_rows"], plan["wavefronts"], plan["join"]) == want:
                    print("planned", D, want, counts, G, idle, width, plan, flush=True)
                    return counts, G, idle, width
    pytest.fail(f"no plan with {want}")


def attend_planned(msq, D, counts, G, idle, width, lens):
    """Calls of these sizes, of every type, by sets of trees and any others, each twice in one workspace."""
    P, rng = 64, np.random.default_rng(D + sum(counts) + width)
    table, blocks = scattered(rng, lens, P)
    table = np.concatenate([table, np.full((len(lens), width - table.shape[1]), -1)], 1)
    p = Pair(msq, blocks, 1, D, P, seed=D, fill=float("nan"))
    p.write(table, [0] * len(lens), lens)
    table[0, 1] = -1  # an absent block
    table = np.concatenate([table, np.full((idle, width), -1)])
    q = rng.normal(size=(sum(counts), G, D))
    rest, lens = [np.zeros((0, 0), bool)] * idle, lens + [0] * idle
    # (the workspace of such calls, with a plan's own need within it)
    need = msq.kv_attention_workspace_bytes(p.gpu, sum(counts), G, len(lens), max(counts), width * P)
    assert msq.kv_attention_plan(p.gpu, sum(counts), G, len(lens), width, max(counts), tree=True)["workspace_bytes"] <= need
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
    for sets in ([T.ancestors(random_tree(rng, n)) for n in counts], [rng.random((n, n)) < 0.3 for n in counts]):
        for dtype, out in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.float32)):
            once, again = (attend(msq, p, q, table, lens, sets + rest, dtype=dtype, out=out, workspace=ws) for _ in range(2))
            assert torch.equal(once, again)


ONE, INSIDE, MORE = "none", "inside", "launch"
FEW, SOME = [([3], 4)], [([26, 5], 4), ([70, 64, 33], 4), ([150], 4), ([40], 1), ([512, 300], 4)]
PLANS = [(D, 16, 4, join, shapes) for D in (64, 128, 256) for join in (ONE, INSIDE, MORE) for shapes in (FEW, SOME)] + \
        [(D, 16, 8, join, SOME) for D in (64, 128) for join in (ONE, INSIDE, MORE)] + \
        [(D, 32 * W, W, join, SOME) for D, W in ((64, 4), (64, 8), (128, 4), (128, 8), (256, 4)) for join in (ONE, MORE)]


@pytest.mark.parametrize("D,tile,waves,join,shapes", PLANS)
def test_every_plan(msq, D, tile, waves, join, shapes):
    """Every kernel, workgroup and join that a call by sets can have, named by its plan."""
    counts, G, idle, width = planned(msq, D, shapes, (tile, waves, join))
    lens = [min(width * 64, max(n, m)) for n, m in zip((2900, 1200, 90), counts)]
    attend_planned(msq, D, counts, G, idle, width, lens)


@pytest.mark.parametrize("join", [ONE, MORE])
@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("D,waves", [(64, 4), (64, 8), (128, 4), (128, 8), (256, 4)])
def test_last_rows_of_every_tile(msq, D, waves, G, join):
    """As test_last_rows_of_many, for every kernel for many rows, unsplit and split: none may go unfound."""
    tile = 32 * waves // G
    n = 2 * tile + 5
    counts = [n, tile + 1, tile + max(1, 16 // G), tile + 16 // G + 1, tile + 32 // G, tile + 32 // G + 1, 1, 2, 32 // G, 0]
    shapes = [(counts, G), ([counts[3], counts[4]], G), ([counts[1]], G), ([counts[5]], G)]  # (few sequences: more parts)
    counts, _, idle, width = planned(msq, D, shapes, (32 * waves, waves, join))
    longest = min(width * 64, 2600)
    lens = [min(longest, b) for b in (longest, longest - 70, max(counts), 33 + n, longest - 1, 300 + n, 200, longest, 64, 100)]
    attend_planned(msq, D, counts, G, idle, width, lens[:len(counts)])

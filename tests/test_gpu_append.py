"""kv_append on the GPU: codes and scales bit for bit those of the oracle's write of the oracle's rotated
keys (see test_gpu_rotary.py on fp64 cosines), queries those of rotary()."""
import numpy as np
import pytest

from oracle import msq_rotary as R
from test_gpu_kv import Pair, codes_of, i32, msq, offsets, rounded, scattered  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def append(msq, p, table, first, counts, rot, dtype, q_heads=0, interleaved=False, amplitude=1.0, positions=None,
           uniform=False, count=None, q_dtype=None, spread=1.0):
    """One call on the GPU and in the oracle; checks the queries."""
    off = offsets(counts)
    k, kt = rounded(p.tokens(off[-1], spread), dtype)
    v, vt = rounded(p.tokens(off[-1], spread), dtype)
    f = rot.frequencies.cpu().numpy() if rot else np.zeros(0)
    taken = counts if count is None else [max(0, min(c, n)) for c, n in zip(count, counts)]
    at = np.concatenate([np.arange(c) + s for s, c in zip(first, counts)] + [np.zeros(0)]) if positions is None else positions
    q, qt = rounded(p.rng.normal(size=(off[-1], max(q_heads, 1), p.D)), dtype)
    got = msq.kv_append(p.gpu, kt, vt, i32(table), i32(first), rot, q=qt if q_heads else None,
                        positions=None if positions is None else i32(positions), offset=None if uniform else i32(off),
                        max_count=max(counts, default=0), count=None if count is None else i32(count), q_dtype=q_dtype)
    turned = R.rotate(k, at, f, interleaved, amplitude) if rot else k
    rows = np.concatenate([np.arange(o, o + t) for o, t in zip(off, taken)] + [np.zeros(0, int)]).astype(int)
    p.ref.write(turned[rows], v[rows], np.asarray(table), first, offsets(taken))
    if q_heads:
        want = torch.from_numpy(R.rotate(q, at, f, interleaved, amplitude) if rot else q).to(q_dtype or dtype)
        live = np.concatenate([np.arange(o, o + t) for o, t, s in zip(off, taken, first) if s >= 0] + [np.zeros(0, int)]).astype(int)
        assert torch.equal(got.cpu()[live], want[live])
    else:
        assert got is None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,P,H,part,interleaved", [
    (64, 32, 1, 64, False), (64, 256, 2, 32, True), (128, 64, 3, 128, False), (128, 64, 2, 48, True),
    (128, 256, 2, 128, False), (128, 32, 9, 64, False), (256, 32, 2, 256, True), (256, 256, 1, 256, False),
    (256, 128, 2, 16, False), (256, 256, 2, 240, True)])
def test_bit_exact(msq, D, P, H, part, interleaved, dtype):
    print(f"append D={D} P={P} H={H} part={part} {interleaved} {dtype}", flush=True)
    rng = np.random.default_rng(P + D)
    lens = [1, P - 1, P, P + 1, 3 * P + 5, 0, 2 * P]
    table, blocks = scattered(rng, [n + 8 for n in lens], P)
    p = Pair(msq, blocks, H, D, P, seed=P, fill=1e9)
    rot = msq.Rotary(msq.rotary_frequencies(part, factor=2.0), interleaved, 0.75)
    kw = dict(interleaved=interleaved, amplitude=0.75)
    append(msq, p, table, [0] * 7, lens, rot, dtype, 2 * H, **kw)
    p.check()
    first = list(lens)
    for counts in ([1] * 7, [2, 0, 1, 3, 1, 2, 5]):
        at = [f if i != 2 else -1 for i, f in enumerate(first)]
        append(msq, p, table, at, counts, rot, dtype, H, spread=np.exp(rng.normal() * 2), **kw)
        first = [f + c if a >= 0 else f for f, c, a in zip(first, counts, at)]
        p.check()
    append(msq, p, table, [0, 3, 1, 0, P + 2, 0, P], [1, 2, 1, 4, 3, 1, 9], rot, dtype, 0, **kw)
    p.check()


@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float32])
def test_long_runs_share_turns(msq, q_dtype):
    """So many blocks that a workgroup takes several heads, the last of them fewer."""
    P, H = 32, 7
    lens = [5000, 3333, 17]
    rng = np.random.default_rng(0)
    table, blocks = scattered(rng, lens, P)
    p = Pair(msq, blocks, H, 64, P, seed=1)
    append(msq, p, table, [0, 0, 0], lens, msq.Rotary(msq.rotary_frequencies(64)), torch.bfloat16, 3, q_dtype=q_dtype)
    p.check()


def test_positions_counts_and_no_rotation(msq):
    """Positions of a tree's rows, counts below and past the rows, and rot None."""
    P, H, D = 32, 2, 128
    rng = np.random.default_rng(8)
    table, blocks = scattered(rng, [200, 200, 200], P)
    p = Pair(msq, blocks, H, D, P, seed=2)
    rot = msq.Rotary(msq.rotary_frequencies(D))
    append(msq, p, table, [0, 0, 0], [70, 70, 70], rot, torch.float32, 4, uniform=True)
    p.check()
    counts = [26, 33, 64]
    append(msq, p, table, [70, 70, 70], counts, rot, torch.float32, 4,
           positions=rng.integers(0, 100000, size=sum(counts)))
    p.check()
    append(msq, p, table, [70, 75, 80], counts, rot, torch.float32, 4, count=[3, 0, 1000])
    p.check()
    append(msq, p, table, [73, 70, 90], [5, 5, 5], None, torch.bfloat16, 4, count=[-4, 5, 2])
    p.check()
    a, b = msq.allocate_kv_cache(blocks, H, D, P), msq.allocate_kv_cache(blocks, H, D, P)
    k, v = (torch.randn(210, H, D, device="cuda").bfloat16() for _ in range(2))
    msq.kv_write(a, k, v, i32(table), i32([0, 0, 0]))
    msq.kv_append(b, k, v, i32(table), i32([0, 0, 0]))
    for x, y in zip(msq.kv_read(a, i32(table), i32([0] * 3), total=210), msq.kv_read(b, i32(table), i32([0] * 3), total=210)):
        assert torch.equal(x, y)


def test_source_rows(msq):
    """Rows of k and v by their numbers, also twice the same, out of order and outside (clamped)."""
    P, H, D = 64, 2, 64
    rng = np.random.default_rng(9)
    table, blocks = scattered(rng, [150, 150], P)
    rot = msq.Rotary(msq.rotary_frequencies(32), True)
    p = Pair(msq, blocks, H, D, P, seed=3)
    k, kt = rounded(p.tokens(40), torch.bfloat16)
    v, vt = rounded(p.tokens(40), torch.bfloat16)
    source = np.array([5, 5, 39, 0, -7, 99, 12, 1, 2, 3])
    msq.kv_append(p.gpu, kt, vt, i32(table), i32([60, 0]), rot, offset=i32([0, 7, 10]), source=i32(source),
                  count=i32([6, 9]))
    rows = np.clip(source, 0, 39)
    at = np.array([60, 61, 62, 63, 64, 65, 0, 1, 2])
    rows = np.concatenate([rows[:6], rows[7:]])
    p.ref.write(np.zeros((60, H, D)), np.zeros((60, H, D)), table, [0, -1], [0, 60, 60])  # what stood there before
    p.gpu.k_scale.zero_()
    p.gpu.v_scale.zero_()
    for t in (p.gpu.k_codes, p.gpu.v_codes):
        t.fill_(128)
    msq.kv_append(p.gpu, kt, vt, i32(table), i32([60, 0]), rot, offset=i32([0, 7, 10]), source=i32(source),
                  count=i32([6, 9]))
    p.ref.write(R.rotate(k[rows], at, rot.frequencies.cpu().numpy(), True), v[rows], table, [60, 0], [0, 6, 9])
    p.check()


def test_absent_blocks_strides_and_empty(msq):
    P, H, D = 32, 2, 64
    rot = msq.Rotary(msq.rotary_frequencies(64))
    table = np.array([[0, -1, 99, 3], [2, 1, -5, 1000]])
    p = Pair(msq, 4, H, D, P, seed=4)
    append(msq, p, table, [0, 0], [120, 128], rot, torch.bfloat16, 2)
    p.check()
    # q, k, v as slices of one fused product, and past the table
    fused = torch.randn(10, 2 * H + 4, D, device="cuda").bfloat16()
    a, b = msq.allocate_kv_cache(4, H, D, P), msq.allocate_kv_cache(4, H, D, P)
    t, first = i32([[0, 1]]), i32([58])
    qa = msq.kv_append(a, fused[:, 4:6], fused[:, 6:], t, first, rot, q=fused[:, :4])
    qb = msq.kv_append(b, fused[:, 4:6].contiguous(), fused[:, 6:].contiguous(), t, first, rot, q=fused[:, :4].contiguous())
    assert torch.equal(qa, qb)
    for x, y in zip(msq.kv_read(a, t, first, total=6), msq.kv_read(b, t, first, total=6)):
        assert torch.equal(x, y)
    # in place
    want = qa.clone()
    assert msq.kv_append(b, fused[:, 4:6], fused[:, 6:], t, first, rot, q=fused[:, :4], q_out=fused[:, :4]).data_ptr() == fused.data_ptr()
    assert torch.equal(fused[:, :4], want)
    none = torch.empty(0, H, D, device="cuda")
    assert msq.kv_append(a, none, none, t, first, rot, q=torch.empty(0, 4, D, device="cuda")).shape == (0, 4, D)
    assert msq.kv_append(a, none, none, i32(np.zeros((0, 2))), i32([]), rot) is None


def test_rows_left_alone_and_graph(msq):
    """Query rows outside every sequence and behind count stay; replays follow changed inputs."""
    P, H, D = 64, 2, 128
    rot = msq.Rotary(msq.rotary_frequencies(128))
    cache = msq.allocate_kv_cache(6, H, D, P)
    table = i32([[0, 1], [2, 3], [4, 5]])
    k, v = (torch.randn(9, H, D, device="cuda") for _ in range(2))
    q = torch.randn(9, 4, D, device="cuda")
    out = torch.full_like(q, 7.0)
    msq.kv_append(cache, k, v, table, i32([10, -1, 20]), rot, q=q, q_out=out, offset=i32([1, 3, 5, 8]), count=i32([1, 2, 3]))
    seven = (out == 7).all(-1).all(-1).cpu().numpy()
    assert list(np.flatnonzero(seven)) == [0, 2, 3, 4, 8]
    first, offset = i32([0, 0, 0]), i32([0, 3, 6, 9])
    other = msq.allocate_kv_cache(6, H, D, P)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        msq.kv_append(cache, k, v, table, first, rot, q=q, offset=offset, max_count=3)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = msq.kv_append(cache, k, v, table, first, rot, q=q, offset=offset, max_count=3)
    msq.kv_append(other, k, v, table, first, rot, offset=offset, max_count=3)
    for step in range(5):
        first += 3
        for t in (k, v, q):
            t.copy_(torch.randn_like(t))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = msq.kv_append(other, k, v, table, first, rot, q=q, offset=offset, max_count=3)
        assert torch.equal(y, want), step
        n = int(first[0]) + 3
        for x, w in zip(msq.kv_read(cache, table, i32([0] * 3), total=3 * n), msq.kv_read(other, table, i32([0] * 3), total=3 * n)):
            assert torch.equal(x, w), step


def heads_a_workgroup(D, P, H, batch, most, width):
    """Heads that a workgroup of keys takes, by the rule at launch_append (msq_kv_append.hip)."""
    strips, lists = P // 32, batch * min((most + P - 2) // P + 1, width)
    waves = strips * (D // (64 if D == 64 or (most >= 16 and strips * (D // 64) <= 16) else 128))
    return min(max(lists * H * waves // (12 * 256), 1), H)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,P,H,batch,tokens,part,interleaved", [
    (64, 32, 7, 256, 40, 64, False), (128, 64, 5, 64, 100, 96, True), (128, 128, 7, 40, 200, 128, False),
    (256, 64, 5, 48, 90, 256, False), (128, 64, 5, 700, 9, 128, False)])
def test_heads_of_a_workgroup(msq, D, P, H, batch, tokens, part, interleaved, dtype):
    """Keys whose workgroups take from one to all of the heads one after another, the last of them fewer: the
    blocks that a call may reach (its max_count, which may be larger than any sequence) make that
    many workgroups.  Rows from a block's start, and behind earlier ones whose codes move."""
    rng = np.random.default_rng(D + P + H)
    width = 64
    rot = msq.Rotary(msq.rotary_frequencies(part), interleaved)
    f = rot.frequencies.cpu().numpy()
    lens = [int(n) for n in rng.integers(tokens // 2, tokens + 1, size=batch)]
    more = [int(n) for n in rng.integers(0, tokens + 1, size=batch)]
    table, blocks = scattered(rng, [a + b for a, b in zip(lens, more)], P)
    table = np.concatenate([table, np.full((batch, width - table.shape[1]), -1)], 1)
    p = Pair(msq, blocks, H, D, P, seed=D)
    writes = []
    for first, counts, spread in (([0] * batch, lens, 1.0), (lens, more, 3.0)):
        k, kt = rounded(p.tokens(sum(counts), spread), dtype)
        v, vt = rounded(p.tokens(sum(counts), spread), dtype)
        off = offsets(counts)
        at = np.concatenate([np.arange(n) + s for s, n in zip(first, counts)])
        p.ref.write(R.rotate(k, at, f, interleaved), v, table, first, off)
        writes.append((kt, vt, i32(first), i32(off), max(counts)))
    met, want = set(), None
    held = lambda: (p.gpu.k_codes, p.gpu.v_codes, p.gpu.k_scale, p.gpu.v_scale)
    for blocks_reached in (0, 2, 4, 6, 8, 12, 17, 26, 34, 64):
        mosts = [max(w[4], min(blocks_reached * P, len(w[0]))) if tokens >= 16 else w[4] for w in writes]
        heads = [heads_a_workgroup(D, P, H, batch, most, width) for most in mosts]
        print(f"heads D={D} P={P} of {H}: {heads} at max_count {mosts}", flush=True)
        for t in held():
            t.fill_(7)
        for (kt, vt, first, off, _), most in zip(writes, mosts):
            msq.kv_append(p.gpu, kt, vt, i32(table), first, rot, offset=off, max_count=most)
        if want is None:
            p.check()  # against the oracle; the others against this one
            want = [t.clone() for t in held()]
        assert all(torch.equal(a, b) for a, b in zip(held(), want))
        met.update(heads)
        if tokens < 16:
            break
    assert any(1 < n < H and H % n for n in met), met

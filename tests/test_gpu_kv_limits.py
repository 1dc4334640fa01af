"""The 8-bit key/value cache on the GPU at the limits of its inputs, against the numpy oracle
and, where scores are so large that only the top ones count, against what is left of the
softmax.  Helpers and error bounds: test_gpu_kv.py."""
import numpy as np
import pytest

from oracle import msq_kv as O
from test_gpu_kv import Pair, crowd, i32, msq, offsets, rounded  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def ways(H, G, D, P, table, L, n, window=0):
    """(kv_attention's block table, kv_len, counts) of one sequence with n query rows, alone and
    so that the work is split; for more than 64 rows of a head also so that the kernel for
    many rows takes it, unsplit and split."""
    wide = lambda w: np.concatenate([table, np.full((1, w), -1)], 1)
    yield table, [L], [n]
    yield wide(400), [L], [n]
    if n * G > 64:
        yield crowd(H, G, D, P, table, [L], [n], window)
        if not window:
            yield wide(450_000_000 // (H * -(-n * G // 16) * 2 * D * P) + 1), [L], [n]


# ---------------------------------------------------------------- scores of any finite size

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size", [5e3, 2.0 ** 19, 3e8, 1e9, 1e12, 1e20, 1e30, 1e37])
def test_attention_scores_of_any_size(msq, D, size):
    """Scores of +-size times code / 127, two tokens level at the top and the others so far below
    that only these two count: the result is the mean of their values within the rounding of
    two weights to f16 (2^-11) and of their exponents (2 x 2^-13 ln 2 while one number of at
    most 2^11 is their reference), lse their score + ln 2.  One of the two may be of a block
    of zeros.  The top is the largest, the least negative, or 0 among huge negative ones."""
    P, L, H, G = 32, 96, 1, 2
    rng = np.random.default_rng(int(np.log2(size)) + D)
    unit = np.sign(rng.normal(size=D))
    table = np.array([[1, 3, 0]])
    tied = [10, 77]
    for sign, top, others in ((1, 127, (1, 41)), (-1, 64, (90, 127)), (-1, 0, (90, 127))):
        code = rng.integers(*others, size=L)
        if sign < 0:
            code[[0, 33, 65]] = 127  # blocks 0 and 2 have the same scale
        code[tied] = top
        k = (code.astype(np.float32) * (np.float32(1) / np.float32(127)))[:, None, None] * unit
        for zeros in (False, True):
            p = Pair(msq, 4, H, D, P, seed=30)
            v = p.tokens(L) * np.repeat([1.0, 30.0, 1000.0], P)[:, None, None]
            if zeros:
                v[:P] = 0
            p.write(table, [0], [L], torch.float32, k=k, v=v)
            kv, vv = (p.ref.values(name, table[0], 0, L)[tied, 0].astype(np.float64) for name in "kv")
            assert np.array_equal(kv[0], kv[1])
            want = vv.mean(0)
            bound = np.abs(vv).mean(0) * (2.0 ** -11 + 2.0 ** -12 * np.log(2) + 2.0 ** -17) + 1e-37
            for n in (1, 40):
                part = 2.0 ** -rng.integers(0, 3, size=(n, G))
                q, qt = rounded(sign * unit * (size * part / D)[..., None], torch.bfloat16)
                score = q.astype(np.float64) @ kv[0]
                for tb, lens, counts in ways(H, G, D, P, table, L, n):
                    print(f"D={D} size={size:g} {sign} {top} zeros={zeros} n={n} batch={len(lens)} "
                          f"width={np.shape(tb)[1]}", flush=True)
                    got, lse = msq.kv_attention(qt, p.gpu, i32(tb), i32(lens), i32(offsets(counts)),
                                                max_count=n, scale=1.0, causal=False,
                                                out_dtype=torch.float32, return_lse=True)
                    torch.cuda.synchronize()
                    got, lse = got.cpu().numpy(), lse.cpu().numpy()
                    assert (np.abs(got - want) <= bound).all(), (got[0, 0, :4], want[:4])
                    e = np.abs(score) * ((D + 32) * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -11
                    assert (np.abs(lse - (score + np.log(2))) <= e).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_one_token_at_scores_of_any_size(msq, D):
    """A row that sees one token returns its value, whatever its score."""
    P, G = 64, 4
    table = np.array([[2]])
    rng = np.random.default_rng(D)
    p = Pair(msq, 3, 1, D, P, seed=31)
    p.write(table, [0], [1], torch.float32)
    k, v = (p.ref.values(name, table[0], 0, 1)[0, 0].astype(np.float64) for name in "kv")
    bound = np.abs(v) * (2.0 ** -11 + 2.0 ** -18) + 1e-37
    for n in (1, 40):
        q, qt = rounded(rng.normal(size=(n, G, D)) * 10.0 ** rng.uniform(5, 36, size=(n, G, 1)), torch.bfloat16)
        for tb, lens, counts in ways(1, G, D, P, table, 1, n):
            got, lse = msq.kv_attention(qt, p.gpu, i32(tb), i32(lens), i32(offsets(counts)), max_count=n,
                                        scale=0.05, causal=False, out_dtype=torch.float32, return_lse=True)
            torch.cuda.synchronize()
            assert (np.abs(got.cpu().numpy() - v) <= bound).all()
            size = 0.05 * np.abs(q.astype(np.float64)) @ np.abs(k)
            e = size * ((D + 32) * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -16
            assert (np.abs(lse.cpu().numpy() - 0.05 * (q.astype(np.float64) @ k)) <= e).all()


# ---------------------------------------------------------------- fp32 queries

@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_fp32_queries_for_fp32_results(msq, D):
    """Queries whose rounding to f16 moves two scores of some hundreds apart by up to a half: fp32
    results go by 22 bits of the query (2^-22 of each term of a score beside 2 D fp32 sums).
    One token has keys where the rounding is down, one where it is up; others are random."""
    P, L, H, G = 32, 96, 1, 2
    rng = np.random.default_rng(D)
    table = np.array([[2, 0, 1]])
    p = Pair(msq, 3, H, D, P, seed=36)
    k = rng.normal(size=(L, H, D)) * 0.02
    half = np.arange(D) % 2
    k[20, 0], k[70, 0] = half, 1 - half
    p.write(table, [0], [L], torch.float32, k=k)
    kk, vv = (p.ref.values(name, table[0], 0, L) for name in "kv")
    step = p.ref.scale["v"][table[0][np.arange(L) // P]]
    mask = np.ones((1, L), bool)
    moved = 0
    for n in (1, 40):
        up = 1 + 2.0 ** -11 + (2 * half - 1) * 2.0 ** -14   # to 1 + 2^-10 where half, to 1 elsewhere
        q = up * 2.0 ** rng.integers(-2, 1, size=(n, G, 1))
        q, qt = rounded(q, torch.float32)
        scale = 1280.0 / D
        want, wl, absum, size, big = O.attention(q, kk, vv, np.repeat(mask, n, 0), scale, step)
        old, *_ = O.attention(q.astype(np.float16), kk, vv, np.repeat(mask, n, 0), scale, step)
        e = size * (2.0 ** -22 + (2 * D + 32) * 2.0 ** -24) + 2.0 ** -20
        bound = absum * (2 * e + 2.0 ** -11 + 2.0 ** -18 + (L + 64) * 2.0 ** -24)[..., None] \
            + (L * 2.0 ** -31 * 127 * big)[..., None] + 1e-37
        moved += int((np.abs(old - want) > 2 * bound).sum())
        for tb, lens, counts in ways(H, G, D, P, table, L, n):
            got, lse = msq.kv_attention(qt, p.gpu, i32(tb), i32(lens), i32(offsets(counts)), max_count=n,
                                        scale=scale, causal=False, out_dtype=torch.float32, return_lse=True)
            torch.cuda.synchronize()
            assert (np.abs(got.cpu().numpy() - want) <= bound).all(), len(lens)
            lb = e + np.abs(wl) * 2.0 ** -22 + (L + 64) * 2.0 ** -24
            assert (np.abs(lse.cpu().numpy() - wl) <= lb).all()
    assert moved > 100  # what rounded queries give is far outside


# ---------------------------------------------------------------- lengths past the table

@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_length_past_the_table(msq, D):
    """A kv_len past what its table holds: the rows stand at its end all the same, and see those of
    the tokens up to there that the table has."""
    P, G, T = 32, 2, 96
    table = np.array([[2, 0, 1]])
    p = Pair(msq, 3, 1, D, P, seed=32)
    p.write(table, [0], [T], torch.float32)
    rng = np.random.default_rng(D)
    k, v = (p.ref.values(name, table[0], 0, T) for name in "kv")
    for n, L in ((1, 97), (1, 120), (50, 97), (50, 120), (50, 146), (50, 500), (50, 2 ** 31 - 1), (3, 2 ** 31 - 1)):
        q, qt = rounded(rng.normal(size=(n, G, D)), torch.bfloat16)
        pos = L - n + np.arange(n, dtype=np.int64)[:, None]
        for window in (0, 40, 2 ** 31 - 1):
            mask = np.arange(T)[None] <= pos
            if window:
                mask &= np.arange(T)[None] > pos - window
            want, wl, absum, size, big = O.attention(q, k, v, mask, 1 / np.sqrt(D), p.ref.scale["v"][table[0][np.arange(T) // P]])
            e = size * (D + 32) * 2.0 ** -24 + 2.0 ** -20
            bound = absum * (2 * e + 2.0 ** -11 + 2.0 ** -18 + (T + 64) * 2.0 ** -24)[..., None] \
                + (T * 2.0 ** -31 * 127 * big)[..., None] + 1e-37
            calls = [(table, [L], [n])]
            if n * G > 64:
                calls.append(crowd(1, G, D, P, table, [L], [n], window if window < 1000 else 0))
            for tb, lens, counts in calls:
                print(f"D={D} n={n} L={L} window={window} batch={len(lens)}", flush=True)
                got, lse = msq.kv_attention(qt, p.gpu, i32(tb), i32(lens), i32(offsets(counts)), max_count=n,
                                            window=window, out_dtype=torch.float32, return_lse=True)
                torch.cuda.synchronize()
                got, lse = got.cpu().numpy(), lse.cpu().numpy()
                assert (np.abs(got - want) <= bound).all()
                none = ~mask.any(1)
                assert (got[none] == 0).all() and np.isneginf(lse[none]).all() and np.isfinite(lse[~none]).all()
    # nobody is masked without causal
    q, qt = rounded(rng.normal(size=(2, G, D)), torch.bfloat16)
    a = msq.kv_attention(qt, p.gpu, i32(table), i32([T]), causal=False)
    b = msq.kv_attention(qt, p.gpu, i32(table), i32([2 ** 31 - 1]), causal=False)
    c = msq.kv_attention(qt, p.gpu, i32(table), i32([-5]), causal=False)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and not bool(c.any())


# ---------------------------------------------------------------- blocks that nothing was written to

@pytest.mark.parametrize("fill", [float("inf"), float("nan"), 3e38, -1.0])
@pytest.mark.parametrize("D,G", [(64, 3), (128, 2), (256, 2)])
def test_attention_window_over_unwritten_blocks(msq, D, G, fill):
    """A cache whose first blocks were never written (a sequence that came with a window): whatever
    their scales hold, nothing of them is seen."""
    P, L, n, w = 32, 256, 40, 50
    table = np.array([[3, 1, 6, 0, 7, 2, 5, 4]])
    p = Pair(msq, 8, 1, D, P, seed=33, fill=fill)
    first = L - n - w + 1  # 167: in the second half of 64 tokens
    p.write(table, [160], [L - 160], torch.float32)
    assert first // 64 * 64 < 160 <= first
    q, qt = rounded(np.random.default_rng(D).normal(size=(n, G, D)), torch.bfloat16)
    for rows in (1, n):
        for tb, lens, counts in ways(1, G, D, P, table, L, rows, w):
            got, lse = msq.kv_attention(qt[-rows:], p.gpu, i32(tb), i32(lens), i32(offsets(counts)), max_count=rows,
                                        window=w, out_dtype=torch.float32, return_lse=True)
            torch.cuda.synchronize()
            p.close(got, lse, q[-rows:], table[0], L, torch.bfloat16, True, w, 1 / np.sqrt(D))


# ---------------------------------------------------------------- value scales

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("low,high,gap", [(-85, 20, 20), (-85, 105, 20), (-85, 105, 90), (-85, -30, 40),
                                          (-20, 50, 45), (-85, 105, 500), (-85, 105, 3000)])
def test_attention_value_scales_far_apart_under_the_top_scores(msq, D, low, high, gap):
    """Blocks of values near 2^low whose scores are e^gap above those of values near 2^high, up to
    2^190 apart: the error stays relative to the largest contribution, whichever it is, and lse
    is that of the scores; in any order, in one wavefront, in several, and in several parts."""
    P, H, G = 32, 1, 2
    rng = np.random.default_rng(D + gap)
    unit = np.sign(rng.normal(size=D))
    for blocks, lows in ((2, [0]), (2, [1]), (14, [0, 3, 4]), (14, [13]), (14, [0, 1, 2, 3, 5, 6, 8, 9, 10, 11, 12])):
        L = blocks * P
        table = rng.permutation(blocks)[None]
        p = Pair(msq, blocks, H, D, P, seed=34)
        k, v = rng.normal(size=(blocks, P, H, D)) * 0.01, p.tokens(L).reshape(blocks, P, H, D)
        v *= 2.0 ** high
        v[lows] *= 2.0 ** (low - high)
        k[lows] += unit * gap / D
        v = v.clip(-3e38, 3e38)
        p.write(table, [0], [L], torch.float32, k=k.reshape(L, H, D), v=v.reshape(L, H, D))
        for n in (1, 40):
            q = unit + rng.normal(size=(n, G, D)) * 0.01
            for tb, lens, counts in ways(H, G, D, P, table, L, n):
                print(f"D={D} {low} {high} {gap} blocks={blocks} {lows} n={n} batch={len(lens)} "
                      f"width={np.shape(tb)[1]}", flush=True)
                full = np.zeros((sum(counts), G, D))
                full[:n] = q
                p.attend(full, tb, lens, counts, scale=1.0)


# ---------------------------------------------------------------- a cache whose buffers change

def test_cache_that_grows(msq):
    """Buffers set anew between calls are the ones that the next call uses."""
    p = Pair(msq, 2, 2, 64, 32, seed=35)
    p.write([[0, 1]], [0], [64])
    old = p.gpu.k_codes, p.gpu.k_codes.clone()
    k0, v0 = msq.kv_read(p.gpu, i32([[0, 1]]), i32([0]), total=64)
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        t = getattr(p.gpu, name)
        setattr(p.gpu, name, torch.cat([torch.zeros_like(t), t]))
    p.gpu.num_blocks = 4
    k1, v1 = msq.kv_read(p.gpu, i32([[2, 3]]), i32([0]), total=64)
    x = torch.randn(32, 2, 64, device="cuda")
    msq.kv_write(p.gpu, x, x, i32([[1]]), i32([0]))
    q = torch.randn(1, 4, 64, device="cuda")
    a = msq.kv_attention(q, p.gpu, i32([[2, 3]]), i32([64]))
    torch.cuda.synchronize()
    assert torch.equal(k0, k1) and torch.equal(v0, v1)
    assert torch.equal(*old) and bool(p.gpu.k_scale[1].any()) and bool(a.any())


# ---------------------------------------------------------------- the example's workspace

@pytest.mark.parametrize("most", [2049, 2100, 130])
def test_example_with_lengths_inside_a_block(msq, most):
    """The example's decode steps with the workspace that it keeps, sized for tokens that end inside
    a block: 4 sequences, 32 heads on 8 of 128."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import cached_attention as ex
    layer = ex.CachedAttention(128, 32, 8, 128, 4, most)
    layer(torch.randn(4 * 5, 128, device="cuda").bfloat16())
    for _ in range(3):
        x = torch.randn(4, 128, device="cuda").bfloat16()
        y, q, a = layer(x, workspace=layer.workspace)
        own = msq.kv_attention(q, layer.cache, layer.table, layer.length)
        torch.cuda.synchronize()
        assert torch.equal(a, own) and torch.isfinite(y).all()
    assert layer.length.tolist() == [8] * 4


# ---------------------------------------------------------------- many sequences without max_count

@pytest.mark.parametrize("D,P,H,batch,rows", [(64, 32, 1, 4096, 5), (256, 256, 2, 8192, 8)])
def test_write_and_read_without_max_count(msq, D, P, H, batch, rows):
    """Ragged batches that leave max_count to the rows of all sequences, which makes more workgroups
    than one launch of 1024 threads each takes (and, for the second, more than one launch of
    theirs): the same codes, scales and values as with max_count."""
    width = -(-batch * rows // P) + 1
    entry = np.arange(batch) % width
    table = np.full((batch, width), -1)
    table[np.arange(batch), entry] = np.random.default_rng(D).permutation(batch)
    first, table = i32(entry * P + 5), i32(table)
    offset = i32(np.arange(batch + 1) * rows)
    g = torch.Generator(device="cuda").manual_seed(D)
    k, v = (torch.randn(batch * rows, H, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    a, b = (msq.allocate_kv_cache(batch, H, D, P) for _ in range(2))
    for c in (a, b):
        c.k_codes.zero_(), c.v_codes.zero_()
    msq.kv_write(a, k, v, table, first, offset, max_count=rows)
    msq.kv_write(b, k, v, table, first, offset)
    want = msq.kv_read(a, table, first, offset, total=batch * rows, max_count=rows)
    got = msq.kv_read(b, table, first, offset, total=batch * rows)
    torch.cuda.synchronize()
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert float((got[0].float() - k.float()).abs().max()) <= float(a.k_scale.max()) * 0.51 + 2.0 ** -6

"""The 8-bit key/value cache on the GPU against the numpy oracle.

Writing and reading are bit-exact: codes byte by byte in the documented order,
scales, and values.  Attention is checked element by element against fp64
attention over the cache's values, within
    E = 2 e + 2^-11 + 2^-18 + (L + 64) 2^-24,    e = S (r + (D + 32) 2^-24) + 2^-20
times sum_t p_t |v_t|, where S = max_t scale * sum_d |q_d k_td| bounds the scores, r is the
rounding of the query to f16 (0 for bf16 queries, 2^-11 for fp32), 2^-11 is the
rounding of the weights to f16, and the rest fp32 sums over D and L terms; plus
L 2^-31 * 127 max_t p_t s_t for weights below the normal f16 numbers, plus half a
unit in the last place for bf16 outputs.
"""
import numpy as np
import pytest

from oracle import msq_kv as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def msq():
    import block_wise_mixed_amd as m
    m.load_library()
    assert torch.cuda.is_available()
    return m


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def rounded(x, dtype):
    """fp32 array of the values `dtype` holds for x."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype)
    return t.float().numpy(), t.cuda()


def codes_of(cache, name, blocks):
    """Codes [len(blocks)][heads][slot][dim] read byte by byte in the documented order."""
    P, D = cache.block_tokens, cache.head_dim
    raw = (cache.k_codes if name == "k" else cache.v_codes)[blocks].cpu().numpy().astype(np.int32)
    t, d = np.meshgrid(np.arange(P), np.arange(D), indexing="ij")
    return raw[:, :, (O.key_byte if name == "k" else O.value_byte)(t, d, D)] - 128


def offsets(counts):
    return [int(sum(counts[:i])) for i in range(len(counts) + 1)]


class Pair:
    """A cache on the GPU and its oracle, written together."""

    def __init__(self, msq, blocks, H, D, P, seed=0, fill=None):
        self.msq, self.H, self.D = msq, H, D
        self.gpu = msq.allocate_kv_cache(blocks, H, D, P)
        self.ref = O.Cache(blocks, H, D, P)
        self.rng = np.random.default_rng(seed)
        if fill is not None:  # what was never written may hold anything
            for t in (self.gpu.k_codes, self.gpu.v_codes):
                t.copy_(torch.randint(0, 256, t.shape, dtype=torch.uint8))
            self.gpu.k_scale.fill_(fill)
            self.gpu.v_scale.fill_(fill)

    def tokens(self, n, spread=1.0):
        x = self.rng.normal(size=(n, self.H, self.D)) * spread
        x[:, :, :3] *= 6
        return x

    def write(self, table, first, counts, dtype=torch.bfloat16, k=None, v=None, uniform=False):
        off = offsets(counts)
        k, kt = rounded(self.tokens(off[-1]) if k is None else k, dtype)
        v, vt = rounded(self.tokens(off[-1], np.exp(self.rng.normal(size=(off[-1], 1, 1))))
                        if v is None else v, dtype)
        self.msq.kv_write(self.gpu, kt, vt, i32(table), i32(first),
                          None if uniform else i32(off), max_count=max(counts, default=0))
        self.ref.write(k, v, np.asarray(table), first, off)

    def check(self):
        torch.cuda.synchronize()
        blocks = np.flatnonzero(self.ref.written.any(1))
        at = self.ref.written[blocks]
        for name in "kv":
            got = codes_of(self.gpu, name, torch.from_numpy(blocks).cuda())
            want = self.ref.codes[name][blocks]
            got, want = (a.transpose(0, 2, 1, 3)[at] for a in (got, want))
            assert np.array_equal(got, want), name
            scale = (self.gpu.k_scale if name == "k" else self.gpu.v_scale).cpu().numpy()
            assert np.array_equal(scale[blocks].view(np.uint32),
                                  self.ref.scale[name][blocks].view(np.uint32)), name

    def attend(self, q, table, lens, counts, dtype=torch.bfloat16, out=torch.float32, causal=True,
               window=0, scale=0.0, **kw):
        q, qt = rounded(q, dtype)
        off = offsets(counts)
        to = torch.full(qt.shape, float("nan"), dtype=out, device="cuda")  # every row is written
        got, lse = self.msq.kv_attention(qt, self.gpu, i32(table), i32(lens), i32(off),
                                         max_count=max(counts, default=0), scale=scale, causal=causal,
                                         window=window, out=to, return_lse=True, **kw)
        torch.cuda.synchronize()
        table = np.asarray(table)
        for b, (n, L) in enumerate(zip(counts, lens)):
            if not n:
                continue
            sl = slice(off[b], off[b + 1])
            self.close(got[sl], lse[sl], q[sl], table[b], L, dtype, causal, window,
                       scale or 1 / np.sqrt(self.D))
        return got, lse

    def close(self, got, lse, q, row, L, dtype, causal, window, scale, hide=None):
        n, D = q.shape[0], self.D
        t = np.arange(L)
        step = self.ref.scale["v"][row[t // self.ref.P]]
        mask = O.sees(L, n, causal, window)
        if hide is not None:
            mask = mask & ~hide[None, :]
        want, wl, absum, size, big = O.attention(q, self.ref.values("k", row, 0, L),
                                                 self.ref.values("v", row, 0, L), mask, scale, step)
        r = 0.0 if dtype == torch.bfloat16 else 2.0 ** -11
        e = size * (r + (D + 32) * 2.0 ** -24) + 2.0 ** -20
        bound = absum * (2 * e + 2.0 ** -11 + 2.0 ** -18 + (L + 64) * 2.0 ** -24)[..., None] \
            + (L * 2.0 ** -31 * 127 * big)[..., None] + 1e-37
        if got.dtype == torch.bfloat16:
            bound = bound + np.abs(want) * 2.0 ** -8
        got, lse = got.float().cpu().numpy(), lse.cpu().numpy()
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())
        empty = ~mask.any(1)
        assert (got[empty] == 0).all() and np.isneginf(lse[empty]).all()
        full = ~empty
        lb = e + np.abs(wl, where=np.isfinite(wl), out=np.zeros_like(wl)) * 2.0 ** -22 + (L + 64) * 2.0 ** -24
        assert (np.abs(lse[full] - wl[full]) <= lb[full]).all()


def scattered(rng, lens, P, spare=2):
    """Block tables with the blocks of all sequences in random places."""
    width = max(1, max(-(-n // P) for n in lens))
    ids = rng.permutation(len(lens) * width + spare)[:len(lens) * width]
    return ids.reshape(len(lens), width), len(lens) * width + spare


# ---------------------------------------------------------------- write

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,P,H", [(64, 32, 1), (64, 256, 2), (128, 64, 3), (128, 128, 2),
                                   (256, 32, 2), (256, 256, 1)])
def test_write_bit_exact(msq, D, P, H, dtype):
    """Runs that start and end anywhere in a block, empty and skipped sequences, then single
    tokens and short runs on top, whose magnitudes sometimes make the scale grow."""
    print(f"write D={D} P={P} H={H} {dtype}", flush=True)
    rng = np.random.default_rng(P + D)
    lens = [1, P - 1, P, P + 1, 3 * P + 5, 0, 2 * P]
    table, blocks = scattered(rng, [n + 8 for n in lens], P)
    p = Pair(msq, blocks, H, D, P, seed=P, fill=1e9)
    p.write(table, [0] * 7, lens, dtype)
    p.check()
    first = list(lens)
    for counts in ([1] * 7, [2, 0, 1, 3, 1, 2, 5]):
        n = sum(counts)
        grow = np.exp(rng.normal(size=(n, 1, 1)) * 2)
        at = [f if i != 2 else -1 for i, f in enumerate(first)]
        p.write(table, at, counts, dtype, k=p.tokens(n) * grow, v=p.tokens(n) * grow)
        first = [f + c if a >= 0 else f for f, c, a in zip(first, counts, at)]
        p.check()
    # going back into a block (dropped tokens) and to its start (begun anew)
    p.write(table, [0, 3, 1, 0, P + 2, 0, P], [1, 2, 1, 4, 3, 1, 9], dtype)
    p.check()


def test_write_token_by_token(msq):
    """A decode loop: one token a call, every scale growth in between."""
    p = Pair(msq, 4, 2, 128, 32, seed=3)
    table = [[2, 0], [1, 3]]
    for t in range(40):
        p.write(table, [t, t], [1, 1], torch.float32, k=p.tokens(2) * (1 + t % 5), uniform=True)
    p.check()


def test_write_special_values(msq):
    """NaN -> 0, infinities -> +-127, a block of zeros, subnormal and huge magnitudes."""
    p = Pair(msq, 6, 1, 64, 32, seed=4)
    x = p.tokens(6 * 32).astype(np.float32).reshape(6, 32, 1, 64)
    x[0, 3, 0, :4] = [np.nan, np.inf, -np.inf, 2.5]
    x[1] = 0
    x[2] *= 1e-40
    x[3] *= 1e38 / np.abs(x[3]).max()
    x[4] = np.nan
    x[5] = 0
    x[5, 0, 0, 0] = 1e-45
    x = x.reshape(-1, 1, 64)
    p.write([[0, 1, 2, 3, 4, 5]], [0], [6 * 32], torch.float32, k=x, v=-x)
    p.check()
    # zeros first, then something: the scale grows from 0
    p.write([[1]], [1], [1], torch.float32)
    p.check()


def test_write_strided_slices(msq):
    """k and v as slices of one fused product, token-major and head-major."""
    H, D, n = 3, 64, 70
    rng = np.random.default_rng(5)
    qkv = torch.from_numpy(rng.normal(size=(n, 5 * H * D)).astype(np.float32)).cuda()
    k = qkv[:, 3 * H * D:4 * H * D].view(n, H, D)
    v = qkv[:, 4 * H * D:].view(n, H, D)
    table, first = i32([[1, 0, 2]]), i32([5])
    a, b, c = (msq.allocate_kv_cache(3, H, D, 32) for _ in range(3))
    for cache in (a, b, c):
        cache.k_codes.zero_(), cache.v_codes.zero_()
    msq.kv_write(a, k, v, table, first)
    msq.kv_write(b, k.contiguous(), v.contiguous(), table, first)
    hm = lambda t: t.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    msq.kv_write(c, hm(k), hm(v), table, first)
    odd = torch.empty(n * H * D + 1, device="cuda")[1:].view(n, H, D).copy_(k)  # misaligned: copied
    d = msq.allocate_kv_cache(3, H, D, 32)
    d.k_codes.zero_(), d.v_codes.zero_()
    msq.kv_write(d, odd, v, table, first)
    torch.cuda.synchronize()
    for cache in (b, c, d):
        for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
            assert torch.equal(getattr(a, name), getattr(cache, name)), name


def test_write_absent_blocks_and_table_end(msq):
    """Entries outside the cache and positions past the table are dropped; nothing else is
    touched."""
    p = Pair(msq, 4, 2, 128, 32, seed=6)
    for t in (p.gpu.k_codes, p.gpu.v_codes):
        t.fill_(7)
    table = [[0, -1], [99, 2]]
    p.write(table, [0, 0], [64, 64])
    p.write(table, [60, 50], [30, 30])     # runs past the table's 64 positions
    p.check()
    for blk in (1, 3):
        assert bool((p.gpu.k_codes[blk] == 7).all()) and bool((p.gpu.v_codes[blk] == 7).all())
        assert bool((p.gpu.k_scale[blk] == 0).all())


def test_offsets_out_of_range_are_clamped(msq):
    """Broken offsets stay inside the tensors (the values written are unspecified)."""
    c = msq.allocate_kv_cache(4, 1, 64, 32)
    x = torch.ones(8, 1, 64, device="cuda")
    for off in ([-5, 4, 1000], [6, 2, 8], [100, 200, 300]):
        msq.kv_write(c, x, x, i32([[0, 1], [2, 3]]), i32([0, 0]), i32(off))
        k, v = msq.kv_read(c, i32([[0, 1], [2, 3]]), i32([0, 0]), i32(off), total=8)
        o = msq.kv_attention(x, c, i32([[0, 1], [2, 3]]), i32([8, 1 << 30]), i32(off))
    torch.cuda.synchronize()
    assert o.shape == x.shape


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,P,H", [(64, 32, 2), (128, 64, 3), (256, 128, 1), (128, 256, 2)])
def test_read_bit_exact(msq, D, P, H, dtype):
    """Ranges from and to anywhere, empty ones, absent blocks and positions outside the table."""
    print(f"read D={D} P={P} H={H} {dtype}", flush=True)
    rng = np.random.default_rng(D + P)
    lens = [2 * P + 3, 1, 3 * P, 40]
    table, blocks = scattered(rng, lens, P)
    p = Pair(msq, blocks, H, D, P, seed=8, fill=float("nan"))
    p.write(table, [0] * 4, lens, torch.float32)
    lo, hi = [3, 0, P - 1, 40], [2 * P + 1, 1, 3 * P, 40]
    off = offsets([h - l for l, h in zip(lo, hi)])
    k, v = msq.kv_read(p.gpu, i32(table), i32(lo), i32(off), total=off[-1], dtype=dtype)
    torch.cuda.synchronize()
    for name, got in (("k", k), ("v", v)):
        want = np.concatenate([p.ref.values(name, table[b], lo[b], hi[b]) for b in range(4)])
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype)), name
    hole = table.copy()
    hole[0, 1] = -1
    n = 4 * P
    k, v = msq.kv_read(p.gpu, i32(hole[:1]), i32([-5]), None, total=n, dtype=dtype)
    torch.cuda.synchronize()
    pos = np.arange(n) - 5
    gone = (pos < 0) | ((pos >= P) & (pos < 2 * P)) | (pos >= hole.shape[1] * P)
    assert bool((k[torch.from_numpy(gone).cuda()] == 0).all())
    assert bool((v[torch.from_numpy(gone).cuda()] == 0).all())
    want = p.ref.values("v", table[0], 0, P)
    assert torch.equal(v[5:5 + P].cpu(), torch.from_numpy(want).to(dtype))


# ---------------------------------------------------------------- attention

CASES = [  # D, P, H, G, lens, counts
    (64, 32, 2, 1, [1, 2, 31, 32, 33], [1] * 5),
    (128, 64, 1, 4, [64, 65, 127, 500, 1], [1] * 5),
    (128, 64, 2, 8, [1000, 3, 129, 700], [1] * 4),
    (256, 32, 1, 3, [70, 200, 31], [1, 2, 5]),
    (128, 128, 3, 5, [300, 77, 128], [3, 1, 4]),
    (128, 64, 1, 16, [200, 90], [1, 1]),
    (64, 256, 1, 7, [600, 257], [5, 2]),
    (128, 64, 2, 2, [40, 100, 17], [40, 33, 17]),
    (64, 64, 1, 4, [300, 64], [70, 64]),
    (256, 64, 1, 2, [150, 200], [150, 20]),
    (128, 32, 1, 1, [400], [130]),
    (128, 64, 2, 8, [260, 300], [33, 260]),
    (64, 32, 1, 71, [90], [2]),
    # tables past 1024 tokens: the eight-wavefront tiles
    (128, 64, 2, 4, [1500, 300, 1025], [200, 300, 64]),
    (128, 32, 1, 8, [1090, 33], [700, 33]),
    (128, 256, 1, 3, [2700], [90]),
    (64, 128, 1, 2, [1300, 700], [140, 129]),
    (256, 32, 1, 4, [1100], [40]),
]


@pytest.mark.parametrize("window", [0, 1, 50])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(msq, case, window):
    D, P, H, G, lens, counts = CASES[case]
    print(f"attention {CASES[case]} window={window}", flush=True)
    rng = np.random.default_rng(case)
    table, blocks = scattered(rng, lens, P)
    p = Pair(msq, blocks, H, D, P, seed=case, fill=float("nan"))
    p.write(table, [0] * len(lens), lens)
    q = rng.normal(size=(sum(counts), H * G, D)) * 1.5
    p.attend(q, table, lens, counts, window=window)
    p.attend(q, table, lens, counts, window=window, dtype=torch.float32, out=torch.bfloat16)
    if window == 0:
        p.attend(q, table, lens, counts, causal=False, scale=0.2)
        # other splits of the same work
        for hint in (1, 64, 100000):
            p.attend(q, table, lens, counts, max_kv_len=hint)


def test_attention_rows_that_see_nothing(msq):
    """Sequences without tokens, and more query rows than tokens, in one call with others."""
    for D, G, counts in ((128, 4, [1, 1, 1, 1]), (64, 2, [5, 7, 3, 4]), (128, 8, [60, 3, 90, 64])):
        lens = [0, 3, 0, 33]
        table, blocks = scattered(np.random.default_rng(1), [64] * 4, 64)
        p = Pair(msq, blocks, 2, D, 64, seed=1, fill=float("nan"))
        p.write(table, [0] * 4, lens)
        q = np.random.default_rng(2).normal(size=(sum(counts), 2 * G, D))
        for window in (0, 2):
            p.attend(q, table, lens, counts, window=window)
            p.attend(q, table, lens, counts, window=window, max_kv_len=100000)
        # a long table: the work is split, and some sequences have no part
        wide = np.concatenate([table, np.full((4, 40), -1, table.dtype)], 1)
        for hint in (0, 600):
            p.attend(q, wide, lens, counts, max_kv_len=hint)


def test_attention_long_split(msq):
    """A long cache in many parts beside short ones; the same bits every time, with the same
    workspace, whatever it holds."""
    D, P, H, G = 128, 64, 1, 4
    lens, counts = [5000, 17, 0, 2100], [1, 1, 1, 1]
    table, blocks = scattered(np.random.default_rng(3), lens, P)
    p = Pair(msq, blocks, H, D, P, seed=3)
    p.write(table, [0] * 4, lens)
    q = np.random.default_rng(4).normal(size=(4, H * G, D)) * 2
    need = msq.kv_attention_workspace_bytes(p.gpu, 4, H * G, 4, 1, table.shape[1] * P)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    a, la = p.attend(q, table, lens, counts, workspace=ws)
    for _ in range(3):
        b, lb = p.attend(q, table, lens, counts, workspace=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_attention_workspace_may_hold_anything(msq):
    """Calls of different shapes share one workspace, whose parts are joined inside the launch or
    by a second one: whatever the last call left, and whatever it held at first, the results
    are those with a workspace of their own, bit for bit."""
    rng = np.random.default_rng(20)
    shapes = [(128, 2, 4, [900, 300, 0], 1), (64, 1, 8, [700], 4), (128, 1, 2, [6000], 1),
              (256, 2, 1, [300, 777], 1), (128, 2, 8, [400, 1000], 2), (128, 1, 8, [900], 30)]
    made = []
    for D, H, G, lens, n in shapes:
        table, blocks = scattered(rng, lens, 64)
        p = Pair(msq, blocks, H, D, 64, seed=D + n)
        p.write(table, [0] * len(lens), lens)
        q = torch.randn(n * len(lens), H * G, D, device="cuda")
        need = msq.kv_attention_workspace_bytes(p.gpu, n * len(lens), H * G, len(lens), n,
                                                table.shape[1] * 64)
        want = msq.kv_attention(q, p.gpu, i32(table), i32(lens))
        made.append((p.gpu, q, i32(table), i32(lens), need, want))
    assert sum(m[4] > 0 for m in made) >= 5
    ws = torch.randint(0, 256, (max(m[4] for m in made),), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        for i in rng.permutation(len(made)):
            gpu, q, table, lens, _, want = made[i]
            got = msq.kv_attention(q, gpu, table, lens, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(got, want), shapes[i]


def test_attention_value_scales_far_apart(msq):
    """Value blocks whose scales differ by 2^80, zero blocks among them: the error stays
    relative to the largest contribution."""
    D, P = 128, 32
    for n, G in ((1, 2), (40, 4)):
        L = 8 * P
        p = Pair(msq, 8, 1, D, P, seed=9)
        v = p.tokens(L) * np.repeat(2.0 ** np.array([0, -40, 20, 3, -60, 0, 10, 1]), P)[:, None, None]
        v[5 * P:6 * P] = 0
        p.write([np.arange(8)], [0], [L], torch.float32, v=v)
        q = np.random.default_rng(n).normal(size=(n, G, D)) * 3
        p.attend(q, [np.arange(8)], [L], [n])
        # only zero blocks and tiny ones
        p.write([np.arange(8)], [0], [L], torch.float32, v=v * 0)
        p.attend(q, [np.arange(8)], [L], [n])
        p.write([np.arange(8)], [0], [L], torch.float32, v=p.tokens(L) * 1e-24)
        p.attend(q, [np.arange(8)], [L], [n])


def test_attention_score_extremes(msq):
    """Scores in the thousands (one token takes all), tiny and huge queries, keys of zeros."""
    D, P, L = 128, 64, 300
    table = [np.arange(5)]
    p = Pair(msq, 5, 2, D, P, seed=10)
    k = p.tokens(L)
    k[64:128] = 0
    p.write(table, [0], [L], torch.float32, k=k)
    rng = np.random.default_rng(11)
    for n in (1, 50):
        for f in (30.0, 1e-30, 1e-42, 1e4):
            p.attend(rng.normal(size=(n, 4, D)) * f, table, [L], [n])
        p.attend(np.zeros((n, 4, D)), table, [L], [n])
        q = rng.normal(size=(n, 4, D)) * 1e30
        p.attend(q, table, [L], [n], scale=1e-30)


def test_attention_ignores_what_is_masked(msq):
    """Slots past a sequence's length, other blocks, absent blocks: whatever they hold."""
    D, P, L = 128, 64, 200
    p = Pair(msq, 6, 1, D, P, seed=12, fill=float("inf"))
    table = np.array([[1, 4, 2, 3]])
    p.write(table, [0], [L])
    rng = np.random.default_rng(13)
    for n in (1, 70):
        q, qt = rounded(rng.normal(size=(n, 4, D)), torch.bfloat16)
        hole = table.copy()
        hole[0, 1] = -7
        for row in (table, hole):
            got, lse = msq.kv_attention(qt, p.gpu, i32(row), i32([L]), out_dtype=torch.float32,
                                        return_lse=True)
            torch.cuda.synchronize()
            hide = (np.arange(L) // P == 1) if row is hole else None
            p.close(got, lse, q, table[0], L, torch.bfloat16, True, 0, 1 / np.sqrt(D), hide)


def test_attention_nonfinite_queries_stay_in_their_rows(msq):
    D, P, L = 128, 64, 300
    p = Pair(msq, 5, 1, D, P, seed=14)
    table = [np.arange(5)]
    p.write(table, [0], [L])
    for n, G in ((1, 4), (2, 8), (60, 4)):
        q = torch.randn(n, G, D, device="cuda")
        good = msq.kv_attention(q, p.gpu, i32(table), i32([L]), out_dtype=torch.float32)
        q2 = q.clone()
        q2[0, 1, 5] = float("nan")
        q2[n - 1, 3, 0] = float("inf")
        q2[n - 1, 2, 0] = -float("inf")
        got = msq.kv_attention(q2, p.gpu, i32(table), i32([L]), out_dtype=torch.float32)
        torch.cuda.synchronize()
        bad = torch.zeros(n, G, dtype=torch.bool)
        bad[0, 1] = bad[n - 1, 3] = bad[n - 1, 2] = True
        assert torch.isnan(got.cpu()[bad]).all()
        assert torch.equal(got.cpu()[~bad], good.cpu()[~bad])


def test_strided_queries_and_given_out(msq):
    D, P, H, G, n = 64, 32, 2, 3, 9
    p = Pair(msq, 4, H, D, P, seed=15)
    table = [np.arange(4)]
    p.write(table, [0], [100])
    qkv = torch.randn(n, (G + 2) * H * D, device="cuda").bfloat16()
    q = qkv[:, :G * H * D].view(n, G * H, D)
    a = msq.kv_attention(q, p.gpu, i32(table), i32([100]))
    out = torch.empty_like(a)
    b = msq.kv_attention(q.contiguous(), p.gpu, i32(table), i32([100]), out=out)
    c = msq.kv_attention(q.permute(1, 0, 2).contiguous().permute(1, 0, 2), p.gpu, i32(table), i32([100]))
    torch.cuda.synchronize()
    assert b is out and torch.equal(a, b) and torch.equal(a, c)


def test_empty_calls(msq):
    c = msq.allocate_kv_cache(2, 1, 64, 32)
    x = torch.empty(0, 1, 64, device="cuda")
    msq.kv_write(c, x, x, i32([[0]]), i32([0]))
    k, v = msq.kv_read(c, i32([[0]]), i32([0]), total=0)
    assert k.shape == v.shape == (0, 1, 64)
    assert msq.kv_attention(x, c, i32([[0]]), i32([0])).shape == (0, 1, 64)
    assert msq.kv_attention(x, c, i32(np.zeros((0, 1))), i32([])).shape == (0, 1, 64)
    torch.cuda.synchronize()


def test_refusals(msq):
    """What does not fit raises, before any launch, and leaves the cache as it is."""
    c = msq.allocate_kv_cache(4, 2, 64, 32)
    c.k_codes.zero_(), c.v_codes.zero_()
    x, q = torch.ones(4, 2, 64, device="cuda"), torch.ones(4, 6, 64, device="cuda")
    table, first = i32([[0, 1]]), i32([0])
    for args in ((x[:, :1], x, table, first), (x, x[:3], table, first), (x, x.bfloat16(), table, first),
                 (x.cpu(), x, table, first), (x, x, table.long(), first), (x, x, table[0], first),
                 (x, x, table, i32([0, 0])), (x, x, table.cpu(), first)):
        with pytest.raises(ValueError):
            msq.kv_write(c, *args)
    with pytest.raises(TypeError):
        msq.kv_write(c, x.half(), x.half(), table, first)
    with pytest.raises(ValueError):
        msq.kv_read(c, table, first)
    with pytest.raises(ValueError):
        msq.kv_read(c, i32([[0], [1]]), i32([0, 0]), total=3)
    lens = i32([4])
    for kw in (dict(out=torch.empty(4, 6, 32, device="cuda")), dict(out=torch.empty(4, 6, 64)),
               dict(out=torch.empty(4, 6, 64, device="cuda"), out_dtype=torch.bfloat16),
               dict(max_kv_len=1 << 70), dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            msq.kv_attention(q, c, table, lens, **kw)
    with pytest.raises(TypeError):
        msq.kv_attention(q, c, table, lens, out_dtype=torch.float16)
    wide = i32(np.zeros((1, 4000)))
    for kw in (dict(window=4, causal=False), dict(window=-1), dict(scale=-1.0), dict(scale=float("nan")),
               dict(max_kv_len=-1)):
        with pytest.raises(msq.MsqError):
            msq.kv_attention(q, c, table, lens, **kw)
    with pytest.raises(msq.MsqError):                           # 5 query heads on 2
        msq.kv_attention(q[:, :5], c, table, lens)
    with pytest.raises(msq.MsqError):                           # too small for the parts
        msq.kv_attention(q, c, wide, lens, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert not bool(c.k_codes.any()) and not bool(c.k_scale.any())


def test_blocks_past_32_bits_of_bytes(msq):
    """A cache whose code buffers pass 4 GiB, its last blocks in use."""
    P, H, D = 256, 8, 256
    blocks = (1 << 32) // (P * H * D) + 9
    p = Pair(msq, 2, H, D, P, seed=16)
    big = msq.allocate_kv_cache(blocks, H, D, P)
    lens, real = [300], np.array([[blocks - 1, blocks - 7]])
    k, kt = rounded(p.tokens(300), torch.bfloat16)
    v, vt = rounded(p.tokens(300), torch.bfloat16)
    p.ref.write(k, v, np.array([[1, 0]]), [0], [0, 300])
    msq.kv_write(big, kt, vt, i32(real), i32([0]))
    gk, gv = msq.kv_read(big, i32(real), i32([0]), total=300, dtype=torch.float32)
    for n in (1, 40):
        q, qt = rounded(np.random.default_rng(n).normal(size=(n, 2 * H, D)), torch.bfloat16)
        got, lse = msq.kv_attention(qt, big, i32(real), i32(lens), out_dtype=torch.float32, return_lse=True)
        torch.cuda.synchronize()
        p.close(got, lse, q, np.array([1, 0]), 300, torch.bfloat16, True, 0, 1 / 16)
    assert np.array_equal(gk.cpu().numpy(), p.ref.values("k", np.array([1, 0]), 0, 300))
    assert np.array_equal(gv.cpu().numpy(), p.ref.values("v", np.array([1, 0]), 0, 300))


def test_other_stream(msq):
    """A decode loop on a stream that is not the current one; temporaries stay alive on it."""
    D, P, H, G = 128, 64, 2, 4
    p, r = (Pair(msq, 40, H, D, P, seed=17) for _ in range(2))
    table = i32([np.arange(40)])
    side = torch.cuda.Stream()
    xs = [torch.randn(3, H, D + 1, device="cuda")[..., 1:] for _ in range(20)]  # copied by the call
    qs = [torch.randn(3, H * G, D, device="cuda").bfloat16() for _ in range(20)]
    torch.cuda.synchronize()
    outs = []
    for i, (x, q) in enumerate(zip(xs, qs)):
        msq.kv_write(p.gpu, x, x, table, i32([3 * i]), stream=None)
        outs.append(msq.kv_attention(q, p.gpu, table, i32([3 * i + 3])))
    torch.cuda.synchronize()
    lens = [i32([3 * i]) for i in range(21)]
    torch.cuda.synchronize()
    for i, (x, q) in enumerate(zip(xs, qs)):
        msq.kv_write(r.gpu, x, x, table, lens[i], stream=side)
        o = msq.kv_attention(q, r.gpu, table, lens[i + 1], stream=side)
        junk = torch.full((1 << 20,), 3, device="cuda")  # would land in temporaries freed early
        side.synchronize()
        assert torch.equal(o, outs[i])
        del junk


def test_graph_replay(msq):
    """One decode step captured in a HIP graph; lengths and inputs change between replays."""
    D, P, H, G, B = 128, 64, 2, 4, 3
    p, e = (Pair(msq, 60, H, D, P, seed=18) for _ in range(2))
    table = i32(np.arange(60).reshape(3, 20))
    for c in (p, e):
        c.rng = np.random.default_rng(19)
        c.write(table.cpu().numpy(), [0] * 3, [1000, 30, 64])
    k, q = torch.randn(B, H, D, device="cuda"), torch.randn(B, H * G, D, device="cuda")
    first, length = i32([1000, 30, 64]), i32([1001, 31, 65])
    need = msq.kv_attention_workspace_bytes(p.gpu, B, H * G, B, 1, 20 * P)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    out = torch.empty(B, H * G, D, dtype=torch.bfloat16, device="cuda")

    def step(cache):
        msq.kv_write(cache, k, k, table, first)
        msq.kv_attention(q, cache, table, length, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        msq.kv_attention(q, p.gpu, table, first, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(p.gpu)
    for i in range(6):
        k.normal_(), q.normal_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step(e.gpu)
        torch.cuda.synchronize()
        assert torch.equal(got, out), i
        assert torch.equal(p.gpu.k_scale, e.gpu.k_scale)
        first += 1
        length += 1
        torch.cuda.synchronize()


# ---------------------------------------------------------------- many query rows
# A call with more than 64 query rows for a head, whose 16-row tiles would read more than
# 400 MB of cache between them (240 MB for heads of 256), takes another kernel.  Idle sequences beside the small ones
# bring a call there.

def crowd(H, G, D, P, table, lens, counts, window=0, hint=0):
    rows, longest = max(counts) * G, len(table[0]) * P
    if hint:
        longest = min(longest, hint)
    if window:
        longest = min(longest, window + max(counts) + 32)
    assert rows > 64
    more = 450_000_000 // (H * -(-rows // 16) * longest * 2 * D) + 1
    table = np.concatenate([np.asarray(table), np.full((more, len(table[0])), -1)])
    return table, list(lens) + [0] * more, list(counts) + [0] * more


MANY = [(128, 64, 1, 4, [64, 65, 127, 500, 1], [17, 20, 33, 40, 1]),
        (128, 64, 2, 16, [300, 31], [9, 5]),
        (64, 128, 2, 5, [700, 129, 257], [70, 1, 64]),
        (256, 64, 2, 3, [130, 310], [43, 90])] + [c for c in CASES if max(c[5]) * c[3] > 64]


def many_rows(msq, shape, case, window):
    D, P, H, G, lens, counts = shape
    print(f"many rows {shape} window={window}", flush=True)
    rng = np.random.default_rng(100 + case)
    table, blocks = scattered(rng, lens, P)
    p = Pair(msq, blocks, H, D, P, seed=case, fill=float("nan"))
    p.write(table, [0] * len(lens), lens)
    q = rng.normal(size=(sum(counts), H * G, D)) * 1.5
    full = crowd(H, G, D, P, table, lens, counts, window)
    p.attend(q, *full, window=window)
    p.attend(q, *full, window=window, dtype=torch.float32, out=torch.bfloat16)
    if window == 0:
        p.attend(q, *full, causal=False, scale=0.2)
        for hint in (30, 200):  # fewer tokens announced than there are
            p.attend(q, *crowd(H, G, D, P, table, lens, counts, hint=hint), max_kv_len=hint)
        # more tokens than there are: the work is split, and most parts stay empty
        width = 450_000_000 // (len(lens) * H * -(-max(counts) * G // 16) * 2 * D * P) + 1
        wide = np.concatenate([table, np.full((len(lens), width), -1)], 1)
        p.attend(q, wide, lens, counts)


@pytest.mark.parametrize("window", [0, 1, 50])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_attention_many_rows(msq, case, window):
    many_rows(msq, MANY[case], case, window)


@pytest.mark.parametrize("window", [0, 3500])
@pytest.mark.parametrize("shape", [(64, 64, 1, 4, [4000, 333], [64, 50]),
                                   (64, 256, 2, 2, [5000, 600], [127, 128]),
                                   (128, 128, 1, 3, [3333], [85])])
def test_attention_many_rows_long(msq, shape, window):
    """Long sequences: tiles of 256 rows for heads of 64 too."""
    many_rows(msq, shape, 50, window)


@pytest.mark.parametrize("D,P,H,G,lens,counts,window", [
    (128, 64, 8, 4, [8100], [150], 0), (128, 64, 8, 4, [8100], [150], 5000),
    (64, 128, 8, 4, [9000, 3000], [200, 130], 0), (256, 32, 4, 4, [6600, 0], [140, 30], 0)])
def test_attention_many_rows_split(msq, D, P, H, G, lens, counts, window):
    """Long enough for several parts with tokens each; the same bits every time."""
    print(f"many rows split D={D} P={P} lens={lens} window={window}", flush=True)
    table, blocks = scattered(np.random.default_rng(21), lens, P)
    p = Pair(msq, blocks, H, D, P, seed=21, fill=float("nan"))
    p.write(table, [0] * len(lens), lens)
    q = np.random.default_rng(22).normal(size=(sum(counts), H * G, D)) * 1.5
    a, la = p.attend(q, table, lens, counts, window=window)
    b, lb = p.attend(q, table, lens, counts, window=window)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_attention_many_rows_that_see_nothing(msq):
    lens, counts = [0, 3, 0, 33], [60, 3, 90, 64]
    table, blocks = scattered(np.random.default_rng(1), [64] * 4, 64)
    for D, G in ((128, 8), (64, 3), (256, 2)):
        p = Pair(msq, blocks, 2, D, 64, seed=1, fill=float("nan"))
        p.write(table, [0] * 4, lens)
        q = np.random.default_rng(2).normal(size=(sum(counts), 2 * G, D))
        for window in (0, 2):
            p.attend(q, *crowd(2, G, D, 64, table, lens, counts, window), window=window)
        wide = np.concatenate([table, np.full((4, 30000), -1)], 1)
        for hint in (0, 600):
            p.attend(q, wide, lens, counts, max_kv_len=hint)


def test_attention_many_rows_extremes(msq):
    """Value scales far apart, scores in the thousands, tiny and huge queries, keys of zeros."""
    D, P, L, n, G = 128, 32, 256, 40, 4
    table = [np.arange(8)]
    full = crowd(1, G, D, P, table, [L], [n])
    p = Pair(msq, 8, 1, D, P, seed=23)
    v = p.tokens(L) * np.repeat(2.0 ** np.array([0, -40, 20, 3, -60, 0, 10, 1]), P)[:, None, None]
    v[5 * P:6 * P] = 0
    k = p.tokens(L)
    k[64:128] = 0
    rng = np.random.default_rng(24)
    for values in (v, v * 0, p.tokens(L) * 1e-24):
        p.write(table, [0], [L], torch.float32, k=k, v=values)
        for f in (3.0, 30.0, 1e-30, 1e-42, 1e4, 0.0):
            p.attend(rng.normal(size=(n, G, D)) * f, *full)
        p.attend(rng.normal(size=(n, G, D)) * 1e30, *full, scale=1e-30)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gap", [4, 40, 90, 400])
def test_attention_zero_values_under_the_top_scores(msq, D, gap):
    """A block of zero values whose scores are e^gap above all others takes nearly all of the
    softmax; what is left of the other values is still as exact, wherever the block stands."""
    P, L, H, G = 32, 448, 2, 2
    table = [np.arange(14)]
    p = Pair(msq, 14, H, D, P, seed=28)
    rng = np.random.default_rng(29)
    unit = np.sign(rng.normal(size=(H, D)))
    for at in (0, 5, 13):
        k, v = rng.normal(size=(L, H, D)) * 0.3, p.tokens(L) * 1e-3
        k[at * P:(at + 1) * P] += unit * gap / D
        v[at * P:(at + 1) * P] = 0
        v[((at + 4) % 14) * P:((at + 4) % 14 + 1) * P] = 0
        p.write(table, [0], [L], torch.float32, k=k, v=v)
        for n in (1, 40):
            q = (unit[:, None] + rng.normal(size=(n, H, G, D)) * 0.01).reshape(n, H * G, D)
            p.attend(q, table, [L], [n], scale=1.0)
            p.attend(q, table, [L], [n], scale=1.0, max_kv_len=1 << 20)
            if n * G > 64:
                p.attend(q, *crowd(H, G, D, P, table, [L], [n]), scale=1.0)
                wide = np.concatenate([table, np.full((1, 30000), -1)], 1)
                p.attend(q, wide, [L], [n], scale=1.0)


def test_attention_many_rows_ignore_what_is_masked(msq):
    """Slots past a sequence's length, absent blocks, non-finite queries of other rows."""
    D, P, L, n, G = 128, 64, 200, 70, 4
    p = Pair(msq, 6, 1, D, P, seed=25, fill=float("inf"))
    table = np.array([[1, 4, 2, 3]])
    p.write(table, [0], [L])
    q, qt = rounded(np.random.default_rng(26).normal(size=(n, G, D)), torch.bfloat16)
    hole = table.copy()
    hole[0, 1] = -7
    for row in (table, hole):
        full, lens, counts = crowd(1, G, D, P, row, [L], [n])
        call = lambda x: msq.kv_attention(x, p.gpu, i32(full), i32(lens), i32(offsets(counts)),
                                          max_count=n, out_dtype=torch.float32, return_lse=True)
        got, lse = call(qt)
        torch.cuda.synchronize()
        hide = (np.arange(L) // P == 1) if row is hole else None
        p.close(got, lse, q, table[0], L, torch.bfloat16, True, 0, 1 / np.sqrt(D), hide)
        q2 = qt.clone()
        q2[0, 1, 5] = float("nan")
        q2[n - 1, 3, 0] = float("inf")
        other, _ = call(q2)
        torch.cuda.synchronize()
        bad = torch.zeros(n, G, dtype=torch.bool)
        bad[0, 1] = bad[n - 1, 3] = True
        assert torch.isnan(other.cpu()[bad]).all()
        assert torch.equal(other.cpu()[~bad], got.cpu()[~bad])


def test_attention_many_rows_past_32_bits_of_bytes(msq):
    """A cache whose code buffers pass 4 GiB, its last blocks in use."""
    P, H, D, n, L = 256, 8, 256, 40, 300
    blocks = (1 << 32) // (P * H * D) + 9
    p = Pair(msq, 2, H, D, P, seed=27)
    big = msq.allocate_kv_cache(blocks, H, D, P)
    k, kt = rounded(p.tokens(L), torch.bfloat16)
    v, vt = rounded(p.tokens(L), torch.bfloat16)
    p.ref.write(k, v, np.array([[1, 0]]), [0], [0, L])
    table, lens, counts = crowd(H, 2, D, P, [[blocks - 1, blocks - 7]], [L], [n])
    msq.kv_write(big, kt, vt, i32(table[:1]), i32([0]))
    q, qt = rounded(np.random.default_rng(n).normal(size=(n, 2 * H, D)), torch.bfloat16)
    got, lse = msq.kv_attention(qt, big, i32(table), i32(lens), i32(offsets(counts)), max_count=n,
                                out_dtype=torch.float32, return_lse=True)
    torch.cuda.synchronize()
    p.close(got, lse, q, np.array([1, 0]), L, torch.bfloat16, True, 0, 1 / 16)

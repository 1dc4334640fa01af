"""Refusals of the key/value cache entry points, before any launch (no GPU needed)."""
import ctypes

import pytest

import block_wise_mixed_amd as msq

OK, INVALID, SHAPE, SMALL, UNSUP = 0, 1, 2, 5, 7
BASE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return msq.load_library()


def cache(**kw):
    c = msq._KvCache()
    c.num_blocks, c.kv_heads, c.head_dim, c.block_tokens = 100, 8, 128, 64
    c.k_codes, c.v_codes, c.k_scale, c.v_scale = BASE, BASE * 2, BASE * 3, BASE * 4
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def seqs(**kw):
    s = msq._KvSeqs()
    s.batch, s.table_width, s.block_table, s.offset = 4, 16, BASE * 5, BASE * 6
    s.total, s.max_count = 4, 1
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def attn(**kw):
    a = msq._KvAttn()
    a.q, a.q_token_stride, a.q_head_stride, a.q_heads = BASE * 7, 32 * 128, 128, 32
    a.kv_len, a.out, a.causal = BASE * 8, BASE * 9, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_BOTH = [  # what every entry point refuses
    (dict(num_blocks=0), {}, SHAPE), (dict(num_blocks=1 << 31), {}, SHAPE),
    (dict(kv_heads=0), {}, SHAPE), (dict(kv_heads=-1), {}, SHAPE),
    (dict(head_dim=96), {}, UNSUP), (dict(head_dim=0), {}, UNSUP),
    (dict(block_tokens=16), {}, UNSUP), (dict(block_tokens=48), {}, UNSUP),
    (dict(block_tokens=512), {}, UNSUP),
    (dict(k_codes=None), {}, INVALID), (dict(v_codes=BASE + 8), {}, INVALID),
    (dict(k_scale=BASE + 2), {}, INVALID), (dict(v_scale=None), {}, INVALID),
    ({}, dict(batch=-1), SHAPE), ({}, dict(total=-1), SHAPE), ({}, dict(total=1 << 31), SHAPE),
    ({}, dict(table_width=0), SHAPE), ({}, dict(table_width=1 << 25), SHAPE),
    ({}, dict(max_count=-1), SHAPE), ({}, dict(offset=None, total=5), SHAPE),
    ({}, dict(batch=0, offset=None), SHAPE), ({}, dict(block_table=None), INVALID),
    ({}, dict(block_table=BASE + 1), INVALID), ({}, dict(offset=BASE + 2), INVALID),
]


@pytest.mark.parametrize("c,s,status", BAD_BOTH)
def test_bad_cache_or_sequences(lib, c, s, status):
    c, s = cache(**c), seqs(**s)
    p = BASE * 7
    assert lib.msq_kv_write(c, s, BASE, p, 1024, 128, p, 1024, 128, 0, None) == status
    assert lib.msq_kv_read(c, s, BASE, p, p, 1, None) == status
    assert lib.msq_kv_attention(c, s, attn(), BASE * 10, 1 << 40, None) == status


def test_write_and_read_arguments(lib):
    w, r, p = lib.msq_kv_write, lib.msq_kv_read, BASE * 7
    c, s = cache(), seqs()
    assert w(None, s, BASE, p, 1024, 128, p, 1024, 128, 0, None) == INVALID
    assert w(c, None, BASE, p, 1024, 128, p, 1024, 128, 0, None) == INVALID
    assert w(c, s, None, p, 1024, 128, p, 1024, 128, 0, None) == INVALID
    assert w(c, s, BASE, None, 1024, 128, p, 1024, 128, 0, None) == INVALID
    assert w(c, s, BASE, p, 1024, 128, p + 8, 1024, 128, 0, None) == INVALID
    assert w(c, s, BASE, p, 1024, 128, p, 1024, 128, 2, None) == INVALID
    assert w(c, s, BASE, p, 1020, 128, p, 1024, 128, 0, None) == INVALID   # bf16: multiples of 8
    assert w(c, s, BASE, p, 1024, 128, p, 1024, 126, 1, None) == INVALID   # fp32: multiples of 4
    assert r(c, s, BASE, p, None, 0, None) == INVALID
    assert r(c, s, BASE, p + 4, p, 0, None) == INVALID
    assert r(c, s, BASE, p, p, -1, None) == INVALID
    assert r(None, s, BASE, p, p, 0, None) == INVALID
    # nothing to do: no pointer is looked at
    e = seqs(total=0, block_table=None)
    assert w(c, e, None, None, 0, 0, None, 0, 0, 0, None) == OK
    assert r(c, e, None, None, None, 0, None) == OK
    # more workgroups than a launch takes
    huge = seqs(batch=1 << 20, total=1 << 30, max_count=1 << 30, table_width=1 << 20)
    assert w(c, huge, BASE, p, 1024, 128, p, 1024, 128, 0, None) == SHAPE


def test_attention_arguments(lib):
    f, c, s = lib.msq_kv_attention, cache(), seqs()
    run = lambda ws=BASE * 10, n=1 << 40, s=s, **kw: f(c, s, attn(**kw), ws, n, None)
    assert f(c, s, None, None, 0, None) == INVALID
    assert f(None, s, attn(), None, 0, None) == INVALID
    for kw in (dict(q=None), dict(q=BASE + 8), dict(kv_len=None), dict(out=None), dict(out=BASE + 4),
               dict(q_dtype=3), dict(out_dtype=-1), dict(lse=BASE + 2), dict(q_token_stride=4),
               dict(q_head_stride=-4), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(window=5, causal=0)):
        assert run(**kw) == INVALID, kw
    for kw in (dict(q_heads=0), dict(q_heads=12), dict(window=-1), dict(max_kv_len=-1)):
        assert run(**kw) == SHAPE, kw
    assert run(s=seqs(total=1 << 27, max_count=1 << 27), q_heads=32) == SHAPE  # rows * heads past 2^31
    # a call whose tokens are split needs its workspace
    long = seqs(table_width=4096)
    need = lib.msq_kv_attention_workspace_bytes(c, long, attn())
    assert need >= 4 * 32 * 128 * 4
    assert run(s=long, n=need - 1) == SMALL
    assert run(s=long, ws=None, n=need) == INVALID
    assert run(s=long, ws=BASE + 128, n=need) == INVALID
    assert f(c, seqs(total=0), attn(q=None, out=None), None, 0, None) == OK
    assert f(c, seqs(batch=0, total=0, offset=None), attn(), None, 0, None) == OK


def test_workspace_sizes(lib):
    w, c = lib.msq_kv_attention_workspace_bytes, cache()
    assert w(c, seqs(), None) == 0 and w(None, seqs(), attn()) == 0 and w(c, None, attn()) == 0
    assert w(cache(head_dim=80), seqs(), attn()) == 0
    assert w(c, seqs(total=0), attn()) == 0
    # one short sequence per call: no split, no workspace
    assert w(c, seqs(table_width=1), attn()) == 0
    # a window bounds the tokens that are split
    long = seqs(table_width=1 << 14)
    assert 0 <= w(c, long, attn(window=128)) < w(c, long, attn())
    # the binding asks for the same
    cc = msq.KVCache.__new__(msq.KVCache)
    cc.block_tokens, cc._desc = 64, c
    assert msq.kv_attention_workspace_bytes(cc, 4, 32, 4, 1, 64 * 4096) == \
        w(c, seqs(table_width=4096), attn(max_kv_len=64 * 4096))


def test_attention_many_sequences(lib):
    """Sizes past one launch are refused without overflow; calls whose parts alone would pass it
    are taken unsplit (then only the missing pointer is left to refuse)."""
    f = lib.msq_kv_attention
    run = lambda c, s, **kw: f(c, s, attn(q=None, **kw), BASE * 10, 1 << 40, None)
    c = cache(kv_heads=64)
    many = seqs(batch=1 << 18, total=1 << 18, max_count=0, table_width=1 << 14)
    assert run(cache(), many) == SHAPE                      # max_count 0: 2^18 rows each
    many.max_count = 1
    assert run(cache(), many) == INVALID
    assert run(c, many, q_heads=64) == SHAPE                # 2^24 workgroups
    many.batch = many.total = 1 << 16
    assert run(c, many, q_heads=64) == INVALID              # 2^22 of 2^13 tiles: unsplit
    assert lib.msq_kv_attention_workspace_bytes(c, many, attn(q_heads=64)) == 0
    for batch, total, heads in ((2**31 - 1, 1, 2**31 - 1), (2**31 - 1, 2**31 - 1, 1), (1, 1, 2**31 - 1),
                                (2**23, 2**23, 1), (1, 2**31 - 1, 1)):
        s = seqs(batch=batch, total=total, max_count=0, table_width=1 << 24)
        assert run(cache(kv_heads=heads), s, q_heads=heads) in (SHAPE, INVALID)


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        msq.allocate_kv_cache(4, 1, 96, 64, device="cpu")
    with pytest.raises(ValueError):
        msq.allocate_kv_cache(4, 1, 64, 16, device="cpu")
    with pytest.raises(ValueError):
        msq.allocate_kv_cache(0, 1, 64, 32, device="cpu")
    c = msq.allocate_kv_cache(4, 2, 64, 32, device="cpu")
    assert c.nbytes == 2 * 4 * 2 * 32 * 64 + 2 * 4 * 2 * 4
    x = torch.zeros(3, 2, 64)
    dev = -1
    assert msq._kv_rows(x, "k", 2, 64, dev) == (x, 3, x.data_ptr(), 128, 64, 1)
    for bad in (x[:, :1], x[..., :32], x[0]):
        with pytest.raises(ValueError):
            msq._kv_rows(bad, "k", 2, 64, dev)
    with pytest.raises(TypeError):
        msq._kv_rows(x.double(), "k", 2, 64, dev)
    t = torch.zeros(3, 2, 65)[..., 1:]
    assert msq._kv_rows(t, "k", 2, 64, dev)[0].is_contiguous()
    with pytest.raises(ValueError):
        msq._kv_rows(x, "k", 2, 64, 0)                          # another device
    table = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        msq._kv_seqs(c, table[0], None, 2, 0)
    with pytest.raises(ValueError):
        msq._kv_seqs(c, table, None, 3, 0)                      # 3 rows over 2 sequences
    with pytest.raises(ValueError):
        msq._kv_seqs(c, table.long(), None, 2, 0)
    with pytest.raises(ValueError):
        msq._kv_seqs(c, table, torch.zeros(2, dtype=torch.int32), 2, 0)
    s, keep = msq._kv_seqs(c, table, None, 4, 0)
    assert (s.batch, s.table_width, s.total) == (2, 3, 4)
    assert ctypes.sizeof(msq._KvCache) == 56 and ctypes.sizeof(msq._KvSeqs) == 40

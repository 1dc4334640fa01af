"""Refusals and sizes of the entry points for rotary positions and drafted tokens, before any launch (no
GPU needed)."""
import copy
import ctypes
import pickle

import pytest

import block_wise_mixed_amd as msq
from test_kv_host import BAD_BOTH, attn, cache, seqs

OK, INVALID, SHAPE, SMALL, UNSUP = 0, 1, 2, 5, 7
BASE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return msq.load_library()


def put(s, values):
    for k, v in values.items():
        setattr(s, k, v)
    return s


def rot(**kw):
    r = msq._Rotary()
    r.freq, r.dims, r.amplitude = BASE * 11, 128, 1.0
    return put(r, kw)


def rows(**kw):
    r = msq._RotaryRows()
    r.x, r.x_token_stride, r.x_head_stride = BASE * 12, 32 * 128, 128
    r.out, r.out_token_stride, r.out_head_stride = BASE * 13, 32 * 128, 128
    r.heads, r.head_dim = 32, 128
    return put(r, kw)


def new(q=None, r=None, **kw):
    n = msq._KvNew()
    n.k, n.k_token_stride, n.k_head_stride = BASE * 14, 1024, 128
    n.v, n.v_token_stride, n.v_head_stride = BASE * 15, 1024, 128
    n.kv_rows = 4
    n.rot = rot() if r is None else r
    if q is not None:
        n.q = q
    return put(n, kw)


def draft(**kw):
    d = msq._Draft()
    d.batch, d.offset, d.total, d.max_count, d.vocab = 4, BASE * 16, 20, 5, 1000
    d.tokens, d.parents, d.target, d.target_stride = BASE * 17, BASE * 18, BASE * 19, 1000
    d.draft, d.draft_stride, d.dtype, d.uniform = BASE * 20, 1000, 1, BASE * 21
    d.token, d.taken, d.path = BASE * 22, BASE * 23, BASE * 24
    return put(d, kw)


def test_struct_sizes():
    for struct, fields in ((msq._Rotary, msq._ROTARY), (msq._RotaryRows, msq._ROTARY_ROWS),
                           (msq._KvNew, msq._KV_NEW), (msq._Draft, msq._DRAFT)):
        assert ctypes.sizeof(struct) == fields.size


BAD_ROWS = [(dict(heads=0), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=120), SHAPE),
            (dict(head_dim=1040), SHAPE), (dict(x_dtype=2), INVALID), (dict(out_dtype=-1), INVALID),
            (dict(x=BASE + 8), INVALID), (dict(out=None), INVALID), (dict(out=BASE + 4), INVALID),
            (dict(x_token_stride=4), INVALID), (dict(x_head_stride=-4), INVALID),
            (dict(out_dtype=1, out_head_stride=2), INVALID), (dict(out_token_stride=12), INVALID)]
BAD_ROT = [(dict(freq=None), INVALID), (dict(freq=BASE + 4), INVALID), (dict(dims=8), SHAPE), (dict(dims=-16), SHAPE),
           (dict(dims=120), SHAPE), (dict(dims=144), SHAPE), (dict(amplitude=float("nan")), INVALID),
           (dict(amplitude=float("inf")), INVALID)]


def test_rotary_arguments(lib):
    f = lib.msq_rotary_apply
    p = BASE * 5
    for kw, status in BAD_ROWS + [(dict(x=None), INVALID), (dict(heads=1 << 25), SHAPE)]:
        assert f(rot(), rows(**kw), p, 4, None) == status, kw
    for kw, status in BAD_ROT + [(dict(dims=0), SHAPE)]:
        assert f(rot(**kw), rows(), p, 4, None) == status, kw
    assert f(None, rows(), p, 4, None) == INVALID and f(rot(), None, p, 4, None) == INVALID
    assert f(rot(), rows(), None, 4, None) == INVALID and f(rot(), rows(), p + 2, 4, None) == INVALID
    assert f(rot(), rows(), p, -1, None) == SHAPE and f(rot(), rows(), p, 1 << 31, None) == SHAPE
    assert f(rot(), rows(x=None, out=None), None, 0, None) == OK
    assert f(rot(), rows(heads=1 << 20, head_dim=1024, x_head_stride=1024), p, (1 << 31) - 1, None) == SHAPE


@pytest.mark.parametrize("c,s,status", BAD_BOTH)
def test_append_and_tree_bad_cache_or_sequences(lib, c, s, status):
    c, s = cache(**c), seqs(**s)
    assert lib.msq_kv_append(c, s, BASE, new(kv_rows=1 << 20), None) == status
    assert lib.msq_kv_attention_tree(c, s, attn(), BASE * 7, 1, BASE * 10, 1 << 40, None) == status


def test_append_arguments(lib):
    f, c, s, p = lib.msq_kv_append, cache(), seqs(), BASE
    assert f(c, s, p, None, None) == INVALID
    assert f(c, s, None, new(), None) == INVALID
    for kw, status in [(dict(k=None), INVALID), (dict(v=BASE + 8), INVALID), (dict(dtype=2), INVALID),
                       (dict(k_token_stride=4), INVALID), (dict(v_head_stride=6, dtype=1), INVALID),
                       (dict(kv_rows=3), SHAPE), (dict(kv_rows=1 << 31), SHAPE),
                       (dict(source=BASE, kv_rows=0), SHAPE), (dict(source=BASE + 2), INVALID),
                       (dict(count=BASE + 1), INVALID), (dict(positions=BASE + 3), INVALID)]:
        assert f(c, s, p, new(**kw), None) == status, kw
    for kw, status in BAD_ROT:
        assert f(c, s, p, new(r=rot(**kw)), None) == status, kw
    for kw, status in BAD_ROWS:
        assert f(c, s, p, new(q=rows(**kw)), None) == status, kw
    assert f(c, s, p, new(q=rows(head_dim=64)), None) == SHAPE
    assert f(c, s, p, new(q=rows(), source=BASE), None) == INVALID
    # nothing to do: no pointer is looked at
    assert f(c, seqs(total=0, block_table=None), None, new(k=None, v=None), None) == OK
    assert f(c, seqs(batch=0, total=0, offset=None), None, new(k=None, v=None), None) == OK
    huge = seqs(batch=1 << 20, total=1 << 30, max_count=1 << 30, table_width=1 << 20)
    assert f(c, huge, p, new(kv_rows=1 << 30), None) == SHAPE


def test_draft_tree_arguments(lib):
    f, p = lib.msq_draft_tree, BASE * 3
    call = lambda parents=p, offset=p, batch=4, total=20, most=5, first=p, sets=p, words=1, at=p: f(
        parents, offset, batch, total, most, first, sets, words, at, None)
    for kw, status in [(dict(parents=None), INVALID), (dict(sets=None), INVALID), (dict(parents=p + 1), INVALID),
                       (dict(offset=p + 2), INVALID), (dict(first=p + 3), INVALID), (dict(sets=p + 1), INVALID),
                       (dict(at=p + 2), INVALID), (dict(batch=-1), SHAPE), (dict(total=-1), SHAPE),
                       (dict(total=1 << 31), SHAPE), (dict(most=-1), SHAPE), (dict(words=0), SHAPE),
                       (dict(total=2000, most=33), SHAPE), (dict(total=2000, most=0, words=31), SHAPE),
                       (dict(offset=None, total=21), SHAPE), (dict(offset=None, batch=0), SHAPE),
                       (dict(batch=1 << 25, total=1 << 25, most=1), SHAPE)]:
        assert call(**kw) == status, kw
    assert call(parents=None, sets=None, total=0) == OK
    assert call(offset=None, batch=0, total=0, parents=None) == OK


def test_tree_attention_arguments(lib):
    f, c, s = lib.msq_kv_attention_tree, cache(), seqs()
    run = lambda sets=BASE * 7, words=1, s=s, a=None: f(c, s, a or attn(), sets, words, BASE * 10, 1 << 40, None)
    assert run(sets=None) == INVALID and run(sets=BASE + 2) == INVALID
    assert run(words=0) == SHAPE and run(words=-3) == SHAPE
    assert run(a=attn(causal=0)) == INVALID and run(a=attn(q=None)) == INVALID
    assert f(c, s, None, BASE, 1, None, 0, None) == INVALID and f(c, None, attn(), BASE, 1, None, 0, None) == INVALID
    assert run(sets=None, words=0, s=seqs(total=0)) == OK
    # what a call without sets needs is enough
    long = seqs(table_width=4096)
    need = lib.msq_kv_attention_workspace_bytes(c, long, attn())
    assert f(c, long, attn(), BASE, 1, None, need, None) == INVALID      # (no buffer)
    assert f(c, long, attn(), BASE, 1, BASE * 10, 16, None) == SMALL


def test_verify_arguments(lib):
    f, size = lib.msq_verify_draft, lib.msq_verify_draft_workspace_bytes
    run = lambda ws=BASE, n=1 << 40, **kw: f(draft(**kw), ws, n, None)
    assert f(None, BASE, 1 << 40, None) == INVALID and size(None) == 0
    for kw, status in [(dict(batch=-1), SHAPE), (dict(total=-1), SHAPE), (dict(total=1 << 31), SHAPE),
                       (dict(max_count=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=(1 << 30) + 1), SHAPE),
                       (dict(offset=None, total=21), SHAPE), (dict(target_stride=999), SHAPE),
                       (dict(draft_stride=999), SHAPE), (dict(dtype=2), INVALID), (dict(tokens=None), INVALID),
                       (dict(target=None), INVALID), (dict(token=None), INVALID), (dict(taken=None), INVALID),
                       (dict(path=None), INVALID), (dict(tokens=BASE + 1), INVALID), (dict(parents=BASE + 2), INVALID),
                       (dict(offset=BASE + 3), INVALID), (dict(uniform=BASE + 1), INVALID), (dict(path=BASE + 2), INVALID),
                       (dict(target=BASE + 2), INVALID), (dict(draft=BASE + 1), INVALID),
                       (dict(target=BASE + 1, dtype=0), INVALID), (dict(batch=1 << 25, total=1 << 25), SHAPE),
                       (dict(uniform=None, batch=1 << 20, total=1 << 28, max_count=256), SHAPE)]:
        assert run(**kw) == status, kw
    for kw in (dict(), dict(uniform=None), dict(draft=None),
               dict(vocab=1 << 30, target_stride=1 << 30, draft_stride=1 << 30)):
        need = size(draft(**kw))
        assert need > 0
        assert run(n=need - 1, **kw) == SMALL and run(ws=None, n=need, **kw) == INVALID
        assert run(ws=BASE + 128, n=need, **kw) == INVALID
    assert f(draft(batch=0, offset=None, total=0, token=None, taken=None), None, 0, None) == OK
    assert size(draft(batch=0, offset=None, total=0)) == 0 and size(draft(vocab=0)) == 0
    # 2^32 - 1 threads of one launch: 1024 a sequence between drawn siblings, else 256
    for most, kw in ((1 << 22, dict()), (1 << 24, dict(parents=None)), (1 << 24, dict(draft=None))):
        assert size(draft(batch=most - 1, **kw)) > 0 and size(draft(batch=most, **kw)) == 0
        assert run(batch=most - 1, ws=None, **kw) == INVALID and run(batch=most, ws=None, **kw) == SHAPE


def test_verify_workspace_covers_smaller_calls(lib):
    size = lib.msq_verify_draft_workspace_bytes
    for uniform in (None, BASE):
        for batch in (1, 3, 64, 700, 5000):
            for most in (0, 1, 26, 1024):
                whole = size(draft(batch=batch, total=batch * 26, max_count=most, vocab=200000, uniform=uniform))
                for total in (0, 1, batch, batch * 25):
                    for vocab in (1, 1000, 1024, 5000, 128000, 199999):
                        assert size(draft(batch=batch, total=total, max_count=most, vocab=vocab, uniform=uniform)) <= whole


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    f = msq.rotary_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and f.tolist()[0] == 1.0 and abs(f.tolist()[16] - 0.01) < 1e-15
    half = msq.rotary_frequencies(64, factor=2.0, device="cpu")
    assert torch.equal(half, f / 2)
    parts = msq.rotary_frequencies(64, factor=8.0, original=4096, device="cpu")
    turns = 4096 * f / (2 * torch.pi)
    assert torch.equal(parts[turns >= 32], f[turns >= 32]) and torch.equal(parts[turns <= 1], f[turns <= 1] / 8)
    assert ((parts <= f) & (parts >= f / 8)).all()
    for kw in (dict(dims=63), dict(dims=0), dict(dims=64, base=0), dict(dims=64, factor=-1.0),
               dict(dims=64, original=10, slow=3, fast=2)):
        with pytest.raises(ValueError):
            msq.rotary_frequencies(device="cpu", **kw)
    for bad in (f.float(), f[:7], f[:12], f[::2], f.view(2, 16)):
        with pytest.raises(ValueError):
            msq.Rotary(bad)
    for a in (0.0, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            msq.Rotary(f, amplitude=a)
    r = msq.Rotary(f)
    r.amplitude = 2.0                      # a field set anew reaches the next call
    r.interleaved = True
    assert r.fields()[1] == (f.data_ptr(), 64, 1, 2.0) and r.fields()[2].dims == 64
    r.frequencies = f.float()
    with pytest.raises(ValueError):
        r.fields()
    r = msq.Rotary(f.clone())              # so do a copy's, and data set from outside
    twin = copy.deepcopy(r)
    assert pickle.loads(pickle.dumps(r)).fields()[1][1:] == r.fields()[1][1:]
    assert twin.fields()[1] == (twin.frequencies.data_ptr(), 64, 0, 1.0) != r.fields()[1]
    assert twin.fields()[2].freq == twin.frequencies.data_ptr() != r.fields()[2].freq
    r.frequencies.data = f[:16].clone()
    assert r.fields()[1] == (r.frequencies.data_ptr(), 32, 0, 1.0) and r.fields()[2].dims == 32
    r = msq.Rotary(f)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    x = torch.zeros(2, 2, 64)
    c = msq.allocate_kv_cache(4, 2, 64, 32, device="cpu")
    for call in (lambda: msq.rotary(x, i(0, 1), r), lambda: msq.kv_append(c, x, x, i(0, 1).view(1, 2), i(0), r),
                 lambda: msq.draft_tree(i(-1, 0)), lambda: msq.verify_draft(i(0, 1), torch.zeros(2, 5)),
                 lambda: msq.kv_attention(x, c, i(0, 1).view(1, 2), i(2), tree=i(1, 3).view(2, 1))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError):
        msq.rotary(x[0], i(0, 1), r)
    # rows of a call on drafted tokens
    assert msq._draft_rows(12, None, 3, 0, -1) == (None, 3, 4)
    assert msq._draft_rows(12, i(0, 5, 12), 1, 7, -1)[1:] == (2, 7)
    assert msq._draft_rows(5000, i(0, 5, 5000), 1, 0, -1)[1:] == (2, 1024)
    for args in ((13, None, 3, 0, -1), (5, None, 0, 0, -1), (2050, None, 2, 0, -1), (9, i(0, 9).view(1, 2), 1, 0, -1),
                 (9, i(0, 9).long(), 1, 0, -1), (9, i(0, 9), 1, 1025, -1), (9, i(0, 9), 1, 0, 0)):
        with pytest.raises(ValueError):
            msq._draft_rows(*args)
    for n in (2 ** 31, -1 - 2 ** 31):
        with pytest.raises(ValueError):
            msq.verify_draft_workspace_bytes(4, 2, 100, max_count=n)
    assert msq.verify_draft_workspace_bytes(20, 4, 1000, 5) == lib.msq_verify_draft_workspace_bytes(draft())

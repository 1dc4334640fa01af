"""The Python binding of the key/value cache, without a GPU: its cache object and what it refuses."""
import types

import pytest

import block_wise_mixed_amd as msq

torch = pytest.importorskip("torch")


def make(blocks=4, heads=2, dim=64, tokens=32):
    return msq.allocate_kv_cache(blocks, heads, dim, tokens, device="cpu")


def addresses(c):
    d = c.descriptor()
    return d.num_blocks, d.k_codes, d.v_codes, d.k_scale, d.v_scale


def held(c):
    return (c.num_blocks, c.k_codes.data_ptr(), c.v_codes.data_ptr(), c.k_scale.data_ptr(),
            c.v_scale.data_ptr())


def test_cache_fields_set_anew():
    """A cache that grows: the descriptor follows the fields, and is not made again without need."""
    c = make()
    assert addresses(c) == held(c)
    assert c.descriptor() is c.descriptor()
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        t = getattr(c, name)
        setattr(c, name, torch.cat([t, torch.zeros_like(t)]))
    c.num_blocks = 8
    assert addresses(c) == held(c) and c.descriptor().num_blocks == 8
    assert c.nbytes == 2 * 8 * 2 * 32 * 64 + 2 * 8 * 2 * 4
    old = c.descriptor()
    c.v_scale = c.v_scale.clone()
    assert c.descriptor() is not old and addresses(c) == held(c)


def test_cache_fields_that_do_not_fit():
    c = make()
    good = dict(num_blocks=4, kv_heads=2, head_dim=64, block_tokens=32, k_codes=c.k_codes,
                v_codes=c.v_codes, k_scale=c.k_scale, v_scale=c.v_scale)
    msq.KVCache(**good)
    wide = torch.zeros(4, 2, 2 * 32 * 64, dtype=torch.uint8)
    for bad in (dict(num_blocks=5), dict(kv_heads=3), dict(block_tokens=64), dict(head_dim=128),
                dict(k_codes=c.k_codes[:3]), dict(v_codes=c.v_codes.to(torch.int8)),
                dict(k_scale=c.k_scale[:3]), dict(v_scale=c.v_scale.double()),
                dict(k_codes=wide[..., ::2]), dict(v_scale=torch.zeros(8, 2)[::2]),
                dict(v_codes=c.v_codes.to("meta"))):
        with pytest.raises(ValueError):
            msq.KVCache(**{**good, **bad})
        for name, value in bad.items():
            d = make()
            setattr(d, name, value)
            with pytest.raises(ValueError):
                d.descriptor()
            with pytest.raises(ValueError):
                msq.kv_attention_workspace_bytes(d, 4, 2, 4, 1, 100)


def test_operators_refuse_a_cache_without_a_gpu():
    c = make()
    x, t = torch.zeros(2, 2, 64), torch.zeros(1, 2, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: msq.kv_write(c, x, x, t, n), lambda: msq.kv_read(c, t, n, total=2),
                 lambda: msq.kv_attention(x, c, t, n)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_operators_refuse_a_stream_of_another_device(monkeypatch):
    """A cache that says it is on device 0 (its buffers are never reached) and a stream on 1."""
    c = make()
    monkeypatch.setattr(msq.KVCache, "device", torch.device("cuda", 0))
    c.descriptor()
    c._index = 0
    stream = types.SimpleNamespace(device_index=1, cuda_stream=0)
    x, t = torch.zeros(2, 2, 64), torch.zeros(1, 2, dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: msq.kv_write(c, x, x, t, n, stream=stream),
                 lambda: msq.kv_read(c, t, n, total=2, stream=stream),
                 lambda: msq.kv_attention(x, c, t, n, stream=stream)):
        with pytest.raises(ValueError, match="device 1"):
            call()


def test_sizes_that_do_not_fit_are_refused():
    """Whole numbers past the C structs' fields raise; they do not wrap around."""
    c = make()
    table = torch.zeros(2, 3, dtype=torch.int32)
    for n in (2 ** 32 + 5, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            msq._kv_seqs(c, table, None, 4, n)
        for sizes in ((4, 2, 2, 1, 3, n), (4, 2, n, 1, 3, 1), (4, n, 2, 1, 3, 1)):
            rows, heads, batch, count, entries, window = sizes
            with pytest.raises(ValueError):
                msq.kv_attention_plan(c, rows, heads, batch, entries, count, window=window)
            with pytest.raises(ValueError):
                msq.kv_attention_workspace_bytes(c, rows, heads, batch, count, 100, window=window)
        with pytest.raises(ValueError):
            msq.kv_attention_plan(c, 4, 2, 2, 3, n)
    with pytest.raises(ValueError):
        msq._kv_seqs(c, table, None, 2 ** 64, 0)
    s, _ = msq._kv_seqs(c, table, None, 4, 2 ** 31 - 1)
    assert (s.batch, s.table_width, s.total, s.max_count, s.offset) == (2, 3, 4, 2 ** 31 - 1, None)
    o = torch.tensor([0, 1, 4], dtype=torch.int32)
    s, _ = msq._kv_seqs(c, table, o, 4, 3)
    assert (s.block_table, s.offset) == (table.data_ptr(), o.data_ptr())
    assert msq._KV_SEQS.size <= 40 and msq._KV_ATTN.size <= 88 and msq._KV_CACHE.size == 56
    with pytest.raises(ValueError):
        msq._pack(msq._KV_ATTN, msq._KvAttn(), "scale", 0, 0, 0, 0, 2, 0, 0, "x", 1, 0, 0, 0, 0)

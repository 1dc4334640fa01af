"""Workspace sizes of attention over the key/value cache: one buffer for a maximum serves every
shorter call (no GPU needed)."""
import pytest

import block_wise_mixed_amd as msq
from test_kv_host import attn, cache, lib, seqs  # noqa: F401

# batch, rows of a sequence, kv heads, query heads of each, head dim
SHAPES = [(1, 1, 8, 4, 128), (1, 1, 8, 4, 64), (1, 1, 1, 16, 256), (3, 1, 8, 8, 256), (4, 1, 8, 8, 128),
          (40, 1, 8, 8, 128), (8, 5, 8, 4, 64), (1, 17, 2, 1, 64), (2, 60, 4, 2, 128), (1, 512, 8, 4, 128),
          (1, 2048, 8, 8, 128), (2, 100, 4, 4, 64), (1, 300, 2, 2, 64), (3, 200, 8, 1, 256), (1, 33, 1, 3, 256),
          (7, 130, 5, 3, 64), (1, 4096, 1, 1, 128), (16, 90, 16, 1, 128)]


@pytest.mark.parametrize("shape", SHAPES)
def test_a_buffer_for_the_longest_serves_all(lib, shape):
    batch, n, H, G, D = shape
    c, s, p = cache(kv_heads=H, head_dim=D), seqs(batch=batch, total=batch * n, max_count=n), msq._KvPlan()
    tight = 0
    for window in (0, 700):
        need = most = 0
        for L in [*range(1, 3000, 7), *range(3000, 140000, 331), *range(1 << 20, 1 << 22, 1 << 17)]:
            s.table_width, a = -(-L // 64), attn(q_heads=H * G, max_kv_len=L, window=window)
            assert lib.msq_kv_attention_plan(c, s, a, p) == 0
            need = max(need, p.workspace_bytes)
            # as max_kv_len, or as the table's length where that is not given
            got = lib.msq_kv_attention_workspace_bytes(c, s, a)
            a.max_kv_len = 0
            assert lib.msq_kv_attention_workspace_bytes(c, s, a) >= got >= most
            most = got
            assert got >= need, (L, got, need)
            tight += got <= 1.5 * need
    assert tight > 0 or most == 0


def test_a_buffer_for_the_widest_window_serves_all(lib):
    c, p = cache(), msq._KvPlan()
    for batch, n in ((1, 1), (4, 5), (1, 300)):
        s, need = seqs(batch=batch, total=batch * n, max_count=n, table_width=1 << 14), 0
        for window in [*range(1, 4000, 13), 20000, 100000, 1 << 30, 0]:
            a = attn(window=window)
            assert lib.msq_kv_attention_plan(c, s, a, p) == 0
            need = max(need, p.workspace_bytes)
            assert lib.msq_kv_attention_workspace_bytes(c, s, a) >= need


@pytest.mark.parametrize("batch,H,G,D", [(4, 8, 4, 128), (1, 8, 4, 128), (2, 4, 4, 256), (8, 2, 8, 64)])
def test_binding_size_serves_calls_without_max_kv_len(batch, H, G, D):
    """A buffer for max_kv_len tokens is enough for a call that leaves max_kv_len to the table, which
    ends inside its last block; 2049 tokens with blocks of 64 among them."""
    pytest.importorskip("torch")
    for P in (64, 256):
        c = msq.allocate_kv_cache(1, H, D, P, device="cpu")
        for L in [2049, *range(1, 4200, 5)]:
            size = msq.kv_attention_workspace_bytes(c, batch, H * G, batch, 1, L)
            for given in (0, L, L // 2):
                for ragged in (False, True):
                    plan = msq.kv_attention_plan(c, batch, H * G, batch, -(-L // P), 1, given, ragged=ragged)
                    assert size >= plan["workspace_bytes"], (L, given)

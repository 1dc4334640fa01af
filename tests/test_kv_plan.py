"""Plans of attention over the key/value cache: the query itself (no GPU needed)."""
import ctypes

import pytest

import block_wise_mixed_amd as msq
from test_kv_host import INVALID, OK, SHAPE, UNSUP, attn, cache, lib, seqs  # noqa: F401


def plan_of(lib, c, s, a):
    p = msq._KvPlan()
    assert lib.msq_kv_attention_plan(c, s, a, p) == OK
    return p


def test_plan_refuses(lib):
    f, p = lib.msq_kv_attention_plan, msq._KvPlan()
    assert f(None, seqs(), attn(), p) == INVALID
    assert f(cache(), None, attn(), p) == INVALID
    assert f(cache(), seqs(), None, p) == INVALID
    assert f(cache(), seqs(), attn(), None) == INVALID
    assert f(cache(head_dim=96), seqs(), attn(), p) == UNSUP
    assert f(cache(), seqs(total=-1), attn(), p) == SHAPE
    assert f(cache(), seqs(), attn(q_heads=12), p) == SHAPE
    assert f(cache(), seqs(), attn(window=3, causal=0), p) == INVALID


def test_plan_fields(lib):
    assert ctypes.sizeof(msq._KvPlan) == 24
    e = plan_of(lib, cache(), seqs(total=0), attn())
    assert (e.tile_rows, e.wavefronts, e.parts, e.join, e.workspace_bytes) == (0, 0, 0, 0, 0)
    one = plan_of(lib, cache(), seqs(table_width=1), attn())
    assert (one.tile_rows, one.wavefronts, one.parts, one.join, one.workspace_bytes) == (16, 4, 1, 0, 0)
    inside = plan_of(lib, cache(), seqs(batch=1, total=1, table_width=13), attn())
    assert inside.parts > 1 and inside.join == 1
    long = plan_of(lib, cache(), seqs(table_width=4096), attn())
    assert long.parts > 16 and long.join == 2
    assert long.workspace_bytes >= 4 * 32 * long.parts * (128 * 4 + 8)
    many = plan_of(lib, cache(), seqs(batch=1, total=2048, max_count=2048, table_width=500), attn())
    assert (many.tile_rows, many.wavefronts) == (256, 8)


def test_binding_plan():
    pytest.importorskip("torch")
    c = msq.allocate_kv_cache(1, 8, 128, 64, device="cpu")
    p = msq.kv_attention_plan(c, 1, 32, 1, 13)
    assert p["join"] == "inside" and p["tile_rows"] == 16 and p["workspace_bytes"] > 0
    assert msq.kv_attention_plan(c, 4, 32, 4, 1, ragged=False)["join"] == "none"
    with pytest.raises(msq.MsqError):
        msq.kv_attention_plan(c, 4, 30, 4, 1)


def test_tree_plan(lib):
    f, p = lib.msq_kv_attention_tree_plan, msq._KvPlan()
    assert f(None, seqs(), attn(), p) == INVALID and f(cache(), None, attn(), p) == INVALID
    assert f(cache(), seqs(), None, p) == INVALID and f(cache(), seqs(), attn(), None) == INVALID
    assert f(cache(), seqs(), attn(causal=0), p) == INVALID
    assert f(cache(head_dim=96), seqs(), attn(), p) == UNSUP and f(cache(), seqs(), attn(q_heads=12), p) == SHAPE
    assert f(cache(), seqs(total=0), attn(), p) == OK
    assert (p.tile_rows, p.wavefronts, p.parts, p.join, p.workspace_bytes) == (0, 0, 0, 0, 0)
    # a tree of 26 of one sequence: eight wavefronts, in one part on 751 tokens, in some on 1500
    one = dict(batch=1, total=26, max_count=26)
    for width, parts, join in ((13, 1, 0), (24, 4, 1)):
        assert f(cache(), seqs(table_width=width, **one), attn(), p) == OK
        assert (p.tile_rows, p.wavefronts, p.join) == (16, 8, join) and 1 <= p.parts <= parts
    # within what the size query gives, and as calls without sets where there are no more than 16 rows of a head
    for batch in (1, 3, 40):
        for most in (1, 4, 26, 64, 300):
            for width in (1, 5, 30, 200, 3000):
                s = seqs(batch=batch, total=batch * most, max_count=most, table_width=width)
                other, need = plan_of(lib, cache(), s, attn()), lib.msq_kv_attention_workspace_bytes(cache(), s, attn())
                assert f(cache(), s, attn(), p) == OK and p.workspace_bytes <= need
                if most * 4 <= 16 or other.tile_rows > 16:
                    assert bytes(p) == bytes(other)

"""Large calls of the key/value cache's write and read that one launch does not take: refused only
past their documented size.  Without a GPU a call that is taken ends at its missing device, so
that is asked for no sizes that would be launched on one."""
import pytest

from test_kv_host import BASE, SHAPE, cache, lib, seqs  # noqa: F401


@pytest.mark.parametrize("c,s,write,read", [
    (dict(), dict(batch=1 << 20, total=1 << 30, max_count=1 << 30, table_width=1 << 10), SHAPE, SHAPE),
    (dict(kv_heads=1 << 20), dict(batch=1 << 11, total=1 << 11), SHAPE, SHAPE),
    (dict(kv_heads=64), dict(batch=1 << 20, total=1 << 27, max_count=1 << 20, table_width=17), SHAPE, SHAPE),
])
def test_refused(lib, c, s, write, read):
    c, s, p = cache(**c), seqs(**s), BASE * 7
    assert lib.msq_kv_write(c, s, BASE, p, 1024, 128, p, 1024, 128, 0, None) == write
    assert lib.msq_kv_read(c, s, BASE, p, p, 0, None) == read

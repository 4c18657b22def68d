"""Refusals and empty calls of the paged cache on the host, before anything touches a GPU (CPU
only): the width of a table row, an empty batch, the self-test of the status words."""
import pytest

from tests.test_paged_abi import CALLS, call, desc, host_only, lib  # noqa: F401  (lib: a fixture)


@host_only
@pytest.mark.parametrize("name", CALLS)
def test_table_width(lib, name):  # noqa: F811
    for width in (-1, 5, 1 << 30, -(1 << 31)):
        assert call(lib, name, desc(table_width=width)) == -1, width
        assert b"table_width" in lib.q1m_last_error()
    # what the lengths of a batch may add up to goes by the width (16 of 2^20 entries), not by the pitch
    wide = dict(table_stride=1 << 26, n_kv_heads=4)
    kw = dict(hq=4, batch=2048, stride=512, stride2=512, n=2048, x=None)
    assert call(lib, name, desc(**wide), **kw) == -2
    assert call(lib, name, desc(table_width=16, **wide), **kw) == -1      # the next check: x
    assert b"too large" not in lib.q1m_last_error()


@host_only
def test_fault_selftest_refusals(lib):  # noqa: F811
    for fault, waits in ((0, 1), (-5, 1), (-9, 1), (1, 1), (-8, 0), (-8, 1001)):
        assert lib.q1m_selftest_timeout_behind(fault, waits, 1000, None) == -2


@host_only
@pytest.mark.parametrize("name", CALLS)
def test_an_empty_batch_needs_no_table(lib, name):  # noqa: F811
    assert call(lib, name, desc(page_table=None), batch=0, n=0) == 0
    assert call(lib, name, desc(page_table=None)) == -1

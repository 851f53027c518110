"""Sizes whose counters of 32 bits would pass 2^31 - 1 in the kernels' loops
are refused on the host (no GPU needed): a length of 2^31 - 1 rounded up to
tiles, and steps of up to 16384 past the end of a row, turned negative."""
import pytest

from test_kv_abi import CALLS, attend, cache, evict, lib, table  # noqa: F401

STEP = 16384  # the largest: eight places of four scores for 512 threads


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("page_size,max_pages", [(1, 2 ** 31 - 1), (1, 2 ** 31 - 2 * STEP), (16, 2 ** 27 - 1),
                                                 (1 << 24, 128)])
def test_tables_whose_rows_end_near_2_31(lib, call, page_size, max_pages):  # noqa: F811
    c, t = cache(page_size=page_size), table(max_pages=max_pages, stride=max_pages)
    assert call(lib, c=c, t=t) == -1
    assert b"2^31" in lib.i8q_last_error()


@pytest.mark.parametrize("budget", [2 ** 31 - 1, 2 ** 31 - STEP, 2 ** 31 - 2 * STEP])
def test_budgets_near_2_31(lib, budget):  # noqa: F811
    assert evict(lib, budget=budget) == -1
    assert b"budget" in lib.i8q_last_error()


def test_the_longest_rows_are_taken(lib):  # noqa: F811
    """(A missing workspace is what is left to refuse.)"""
    n = (2 ** 31 - 2 ** 16) // 16
    c = cache(kv_heads=1, page_stride=1024)
    assert attend(lib, c=c, t=table(max_pages=n, stride=n), ws=None) == -1
    assert b"workspace" in lib.i8q_last_error()

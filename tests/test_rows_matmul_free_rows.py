"""The rows that no expert has, as the experts' products number them to write
zeros there, up to the largest number of rows, by the kernel's own arithmetic
on the host (instrumented build)."""
import ctypes

import pytest

import segmented_radix_top_gb300 as st

LARGEST = 2 ** 31 - 257  # rows
WARPS = 152 * 8          # that share the rows: each starts at its own number


@pytest.fixture(scope="module")
def hook():
    return st.load_instrumented().segtopk_test_free_row


@pytest.mark.parametrize("first,end", [(0, 0), (0, 100), (7, 7), (7, 100), (5000, 6000), (0, 2 ** 31 - 1300), (0, LARGEST - 1),
                                       (0, LARGEST), (3, LARGEST), (LARGEST, LARGEST)])
def test_rows_by_number(hook, first, end):
    row = ctypes.c_int64()
    for i in (*range(0, 12), *range(max(first - 3, 0), first + 3), *range(WARPS - 20, WARPS + 3)):
        assert hook(first, end, i, ctypes.byref(row)) == 0
        # numbers past the last one stay past the rows, where nothing is written
        assert row.value == (i if i < first else end + i - first), (i, row.value)


def test_refusals(hook):
    row = ctypes.c_int64()
    for first, end, i in ((-1, 3, 0), (4, 3, 0), (0, 3, -1)):
        assert hook(first, end, i, ctypes.byref(row)) == 1
    assert hook(0, 3, 0, None) == 1
    st.build()
    assert st.load().segtopk_test_free_row(0, 3, 0, ctypes.byref(row)) == 3  # the ordinary build has no such hook

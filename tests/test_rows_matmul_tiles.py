"""The tiles that the experts' products cut an expert's rows into, up to the
largest number of rows, by the kernel's own arithmetic on the host
(instrumented build). No GPU is needed, nor memory for such rows."""
import ctypes

import pytest

import segmented_radix_top_gb300 as st

LARGEST = 2 ** 31 - 257  # rows


@pytest.fixture(scope="module")
def tile():
    L = st.load_instrumented()
    first, width = ctypes.c_int32(), ctypes.c_int32()

    def get(rows, index):
        assert L.segtopk_test_expert_tile(rows, index, ctypes.byref(first), ctypes.byref(width)) == 0, (rows, index)
        return first.value, width.value
    return get


# the sum of the rows and of the tiles, less one, passes 2^31 - 1 from 2139127681 rows on
@pytest.mark.parametrize("rows", [1, 31, 32, 33, 255, 256, 257, 288, 289, 511, 512, 513, 769, 1000, 65537, 2 ** 22 - 1, 2 ** 22,
                                  2 ** 22 + 1, 2 ** 24 + 3, 2 ** 30 + 1, 2139127680, 2139127681, 2139127682, 2 ** 31 - 513,
                                  LARGEST - 1, LARGEST])
def test_tiles_follow_one_another_and_hold_all_rows(tile, rows):
    count = -(-rows // 256)
    step = -(-(-(-rows // count)) // 32) * 32
    at = sorted({i for c in (0, count // 3, count // 2, count) for i in range(c - 40, c + 40) if 0 <= i < count})
    for i in at:
        first, width = tile(rows, i)
        assert first == i * step and 0 < width <= 256, (i, first, width)
        assert width == step if i < count - 1 else first + width == rows, (i, first, width)


def test_every_number_of_rows_up_to_some_tiles(tile):
    for rows in range(1, 1500):
        end = 0
        for i in range(-(-rows // 256)):
            first, width = tile(rows, i)
            assert first == end and 0 < width <= 256
            end += width
        assert end == rows


def test_refusals(tile):
    L = st.load_instrumented()
    n = ctypes.c_int32()
    at = ctypes.byref(n)
    for rows, index in ((0, 0), (-1, 0), (LARGEST + 1, 0), (256, 1), (256, -1)):
        assert L.segtopk_test_expert_tile(rows, index, at, at) == 1
    assert L.segtopk_test_expert_tile(256, 0, None, at) == L.segtopk_test_expert_tile(256, 0, at, None) == 1
    st.build()
    assert st.load().segtopk_test_expert_tile(256, 0, at, at) == 3  # the ordinary build has no such hook

"""Rows in 8 bits against their definition: a scale is two roundings from it,
and a value is the nearest one of x * (448 / a) or, where that product's own
two roundings (2^-23 of it) carry it over the middle between two, the other."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
# the numbers of the type that are not negative
NUMBERS = np.sort(torch.arange(127, dtype=torch.uint8).view(F8).double().numpy())


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def check(x):
    values, scales = st.quantize_rows(x)
    n, width = x.shape
    blocks = -(-width // 128)
    assert values.dtype == F8 and values.shape == (n, width) and scales.dtype == torch.float32 and scales.shape == (n, blocks)
    x, got = ref.f64(x), ref.f64(values)
    full = np.zeros((n, blocks * 128))
    full[:, :width] = np.abs(x)
    most = np.maximum(full.reshape(n, blocks, 128).max(2), 2.0 ** -100)
    assert np.all(np.abs(ref.f64(scales) - most / 448) <= 2.0 ** -24 * most / 448 + 2.0 ** -150)
    want = np.abs(x) * np.repeat(448 / most, 128, 1)[:, :width]
    at = np.searchsorted(NUMBERS, want)
    below, above = NUMBERS[np.maximum(at - 1, 0)], NUMBERS[np.minimum(at, 126)]
    off = np.abs(np.abs(got) - want)
    nearest = np.minimum(np.abs(below - want), np.abs(above - want))
    assert np.all(off <= nearest + 2.1 * 2.0 ** -23 * want)
    assert np.all((np.sign(got) == np.sign(x)) | (got == 0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 16), (3, 127), (3, 128), (5, 129), (64, 2048), (33, 1040), (17, 1001), (700, 640),
                                        (9000, 512), (2, 100000)])
def test_rows(rows, width, dtype):
    check((randn(rows, width, seed=width) * torch.exp(2 * randn(rows, 1, seed=rows))).to(dtype))


def test_strides_and_odd_starts():
    wide = randn(200, 900, seed=1)
    for x in (wide[:, 16:528], wide[:, 3:300], wide[::3, 8:264], wide[:1, :256].expand(200, 256), wide.t()):
        check(x)
        check(x.half()[:, 1:])


def test_zeros_small_and_large_values():
    x = randn(8, 512, seed=1)
    x[0] = 0
    x[1, :128] = 0
    x[2] *= 1e-38   # below the smallest normal number
    x[3] *= 1e-30   # 448 / a, times x, in range; a above 2^-100
    x[4] *= 1e37
    x[5] = torch.tensor([3.4e38, -3.4e38] * 256)
    check(x)
    values, scales = st.quantize_rows(x)
    assert not values[0].float().any() and (scales[0] > 0).all()
    # the largest of a block is 448 unless all are tiny
    assert (values[3:].float().abs().reshape(5, 4, 128).amax(2) == 448).all()


def test_nan_and_infinity_stay_in_their_block():
    x = randn(4, 512, seed=2, dtype=torch.bfloat16)
    clean = st.quantize_rows(x)
    y = x.clone()
    y[1, 130], y[2, 400] = float("nan"), float("inf")
    values, scales = st.quantize_rows(y)
    assert torch.isnan(scales[1, 1]) and torch.isinf(scales[2, 3])
    assert torch.isnan(values.float()[1, 128:256]).all() and torch.isnan(values.float()[2, 400])
    rest = values.float()[2, 384:]
    assert not rest[torch.arange(128, device="cuda") != 16].any()
    same = torch.ones(4, 512, dtype=torch.bool, device="cuda")
    same[1, 128:256] = same[2, 384:] = False
    assert torch.equal(values.float()[same], clean[0].float()[same])


def test_nearest_with_ties_to_even():
    # a block whose largest value is 448: values are taken as they are
    x = torch.zeros(2, 128, device="cuda")
    x[:, 0] = 448
    x[0, 1:8] = torch.tensor([17.0, 19.0, 21.0, 1.0625, 1.1875, 2.0 ** -9 * 0.5, 2.0 ** -9 * 1.5])
    x[1] = -x[0]
    values, scales = st.quantize_rows(x)
    assert torch.equal(scales, torch.ones_like(scales))
    want = torch.tensor([448.0, 16, 20, 20, 1.0, 1.25, 0, 2.0 ** -8], device="cuda")
    assert torch.equal(values.float()[0, :8], want) and torch.equal(values.float()[1, :8], -want)


def test_graph_and_streams():
    x = randn(500, 1000, seed=1, dtype=torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        values, scales = st.quantize_rows(x)
    x.copy_(randn(500, 1000, seed=2, dtype=torch.bfloat16))
    graph.replay()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = st.quantize_rows(x, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(values.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scales, want[1])
    assert st.quantize_rows(x[:0])[1].shape == (0, 8)


def test_past_32_bits():
    x = torch.zeros(600000, 4096, dtype=torch.bfloat16, device="cuda")
    x[-3:] = randn(3, 4096, seed=1, dtype=torch.bfloat16)
    values, scales = st.quantize_rows(x)
    want = st.quantize_rows(x[-3:].clone())
    assert torch.equal(values[-3:].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scales[-3:], want[1])
    assert not values[:3].float().any()

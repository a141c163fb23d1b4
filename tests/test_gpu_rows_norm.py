"""Layer norm and its gradients against their definitions in 64 bits.

Bounds (u = 2^-24): a row's sums go through at most 64 values of a thread, ten
steps over warps and a division, so the mean is off by at most 100 u times the
largest magnitude A of the row; with h the normalised values and r = rstd, h is
off by at most 200 u (1 + A r) (1 + |h|), which covers the mean, the sum of
squares, its root and the products after it."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref

pytestmark = pytest.mark.gpu
U = ref.U32
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
WIDTHS = [1, 7, 8, 64, 65, 128, 256, 511, 520, 1000, 1001, 1024, 1032, 2048, 2049, 2052, 4096, 4100, 5001, 8192, 8200, 16384]


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def inputs(rows, width, dtype, weight_dtype, seed=1):
    x = (randn(rows, width, seed=seed) * torch.exp(randn(rows, 1, seed=seed + 1)) + randn(rows, 1, seed=seed + 2)).to(dtype)
    weight, bias = (1 + 0.2 * randn(width, seed=seed + 3)).to(weight_dtype), randn(width, seed=seed + 4, dtype=weight_dtype)
    return x, weight, bias, randn(rows, width, seed=seed + 5, dtype=dtype)


def statistics(x, eps):
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    return mean, rstd, (x - mean) * rstd


def forward_matches(got, x, weight, bias, eps):
    out, mean_got, rstd_got = got
    xd, w = x.double(), weight.double()
    mean, rstd, h = statistics(xd, eps)
    most = xd.abs().amax(1, keepdim=True)
    ref.within(mean_got, mean[:, 0].cpu().numpy(), (100 * U * most)[:, 0].cpu().numpy())
    ref.within(rstd_got, rstd[:, 0].cpu().numpy(), (200 * U * (1 + most * rstd) * rstd)[:, 0].cpu().numpy())
    want = h * w + (bias.double() if bias is not None else 0)
    bound = 200 * U * (1 + most * rstd) * (1 + h.abs()) * w.abs() + 2 * U * want.abs()
    if bias is not None:
        bound = bound + 2 * U * bias.double().abs()
    assert out.dtype == x.dtype
    ref.within(out, want.cpu().numpy(), (bound + ref.rounded(x.dtype, want.abs())).cpu().numpy())


def gradients(grad, x, weight, eps):
    """In 64 bits, and what bounds a computation of them in 32."""
    g, xd, w = grad.double(), x.double(), weight.double()
    _, rstd, h = statistics(xd, eps)
    gw = g * w
    grad_x = rstd * (gw - gw.mean(1, keepdim=True) - h * (gw * h).mean(1, keepdim=True))
    off = 200 * U * (1 + xd.abs().amax(1, keepdim=True) * rstd) * (1 + h.abs().amax(1, keepdim=True))  # of h and r
    size = gw.abs() + gw.abs().mean(1, keepdim=True) + (1 + h.abs()) * (gw.abs() * (1 + h.abs())).mean(1, keepdim=True)
    n = x.shape[0] + 8
    return ((grad_x, rstd * size * (100 * U + 2 * off)),
            ((g * h).sum(0), (g.abs() * (h.abs() * n * U + off)).sum(0)),
            (g.sum(0), n * U * g.abs().sum(0)))


def check(x, weight, bias, grad, eps=1e-5):
    got = st.layer_norm(x, weight, bias, eps=eps)
    forward_matches(got, x, weight, bias, eps)
    back = st.layer_norm_backward(grad, x, weight, got[1], got[2])
    assert back[0].dtype == x.dtype and back[1].dtype == back[2].dtype == weight.dtype
    for value, (want, bound) in zip(back, gradients(grad, x, weight, eps)):
        ref.within(value, want.cpu().numpy(), (bound + ref.rounded(value.dtype, want.abs())).cpu().numpy())
    return got, back


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dtype):
    check(*inputs(37, width, dtype, dtype))


@pytest.mark.parametrize("rows", [1, 2, 8, 9, 151, 152, 153, 1237, 4864, 4865])
@pytest.mark.parametrize("width", [64, 600, 1024, 2048, 4096])
def test_rows(rows, width):
    check(*inputs(rows, width, torch.bfloat16, torch.float32))


@pytest.mark.parametrize("dtype,weight_dtype", [(torch.bfloat16, torch.float32), (torch.float16, torch.float32),
                                                (torch.float32, torch.float32)])
def test_weight_types_and_no_bias(dtype, weight_dtype):
    for width in (96, 1000, 4096):
        x, weight, _, grad = inputs(50, width, dtype, weight_dtype)
        check(x, weight, None, grad)


def test_strides_and_odd_starts():
    wide = randn(300, 700, seed=3)
    grads = randn(300, 700, seed=4)
    for x, g in ((wide[:, 8:520], grads[:, :512]), (wide[:, 3:204], grads[:, 5:206]), (wide[::2, 100:356], grads[1::2, 100:356]),
                 (wide[:1, :256].expand(300, 256), grads[:1, 64:320].expand(300, 256)), (wide.t(), grads.t())):
        _, weight, bias, _ = inputs(1, x.shape[1], torch.float32, torch.float32)
        check(x, weight, bias, g)
        check(x.bfloat16()[:, 1:], weight[1:], bias[1:], g.bfloat16()[:, 1:])
    base = randn(100 * 64 + 1, seed=5, dtype=torch.bfloat16)
    _, weight, bias, grad = inputs(100, 64, torch.bfloat16, torch.bfloat16)
    check(base[1:].view(100, 64), weight, bias, grad)
    check(base[:-1].view(100, 64), torch.cat([weight, weight])[3:67], bias, grad)


def test_offsets_much_larger_than_the_spread():
    # the mean is 1000 times the deviation: a variance by differences of squares would be lost
    x, weight, bias, grad = inputs(64, 1536, torch.float32, torch.float32)
    check(x * 0 + 1000 + randn(64, 1536, seed=9), weight, bias, grad)
    check(x * 0 - 1000 + randn(64, 1536, seed=9), weight, bias, grad)


def test_values_that_are_all_alike_and_eps():
    x, weight, bias, grad = inputs(20, 640, torch.float32, torch.float32)
    same = torch.full_like(x, 3.0)
    out, mean, rstd = st.layer_norm(same, weight, bias, eps=1e-2)
    # 3 times any count, and its sums, are exact here
    assert torch.equal(mean, torch.full_like(mean, 3)) and torch.equal(out, bias.expand_as(out))
    assert torch.allclose(rstd, torch.full_like(rstd, 10), rtol=1e-6)
    check(x, weight, bias, grad, eps=0.0)
    check(x, weight, bias, grad, eps=10.0)


def test_nan_and_infinity_stay_in_their_row():
    x, weight, bias, grad = inputs(40, 1000, torch.float32, torch.float32)
    got = st.layer_norm(x, weight, bias)
    y = x.clone()
    y[7, 999], y[20, 0] = float("nan"), float("inf")
    bad = st.layer_norm(y, weight, bias)
    keep = [i for i in range(40) if i not in (7, 20)]
    for a, b in zip(got, bad):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(bad[0][7]).all() and torch.isnan(bad[0][20]).all()
    grad_x = st.layer_norm_backward(grad, y, weight, bad[1], bad[2])[0]
    assert torch.equal(grad_x[keep], st.layer_norm_backward(grad, x, weight, got[1], got[2])[0][keep])


def test_gradients_against_differences():
    x, weight, bias, grad = inputs(30, 200, torch.float32, torch.float32)
    got = st.layer_norm(x, weight, bias)
    back = st.layer_norm_backward(grad, x, weight, got[1], got[2])
    g, xd, w, b = (t.double() for t in (grad, x, weight, bias))

    def loss(xd, w, b):
        return (g * (statistics(xd, 1e-5)[2] * w + b)).sum()
    dx, dw, db = (randn(*t.shape, seed=20 + i).double() for i, t in enumerate((x, weight, bias)))
    step = 1e-4  # of a difference whose own error is of its second power: 1e-8 of the third derivative
    for value, (want, bound), d, change in zip(back, gradients(grad, x, weight, 1e-5), (dx, dw, db),
                                               (lambda s: (xd + s * dx, w, b), lambda s: (xd, w + s * dw, b),
                                                lambda s: (xd, w, b + s * db))):
        slope = (loss(*change(step)) - loss(*change(-step))) / (2 * step)
        off = ((bound + ref.rounded(torch.float32, want.abs())) * d.abs()).sum()
        assert abs(float((value.double() * d).sum() - slope)) <= float(off) + 1e-5 * float((want * d).abs().sum())


def test_no_rows():
    weight = torch.ones(64, device="cuda")
    x = torch.zeros(0, 64, device="cuda")
    out, mean, rstd = st.layer_norm(x, weight, weight)
    assert out.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    grad_x, grad_weight, grad_bias = st.layer_norm_backward(x, x, weight, mean, rstd)
    assert grad_x.shape == (0, 64) and not grad_weight.any() and not grad_bias.any()


def test_repeats_streams_and_graphs():
    x, weight, bias, grad = inputs(3000, 1600, torch.bfloat16, torch.bfloat16)
    first = st.layer_norm(x, weight, bias)
    back = st.layer_norm_backward(grad, x, weight, first[1], first[2])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            y = st.layer_norm(x, weight, bias, stream=s)
            got.append((y, st.layer_norm_backward(grad, x, weight, y[1], y[2], stream=s)))
    torch.cuda.synchronize()
    for y, b in got:
        assert all(torch.equal(p, q) for p, q in zip((*y, *b), (*first, *back)))
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = st.layer_norm(x, weight, bias, out=out)
        captured_back = st.layer_norm_backward(grad, x, weight, captured[1], captured[2])
    x.copy_(inputs(3000, 1600, torch.bfloat16, torch.bfloat16, seed=50)[0])
    graph.replay()
    want = st.layer_norm(x, weight, bias)
    assert all(torch.equal(p, q) for p, q in zip(captured, want)) and captured[0] is out
    assert all(torch.equal(p, q) for p, q in zip(captured_back, st.layer_norm_backward(grad, x, weight, want[1], want[2])))


def test_past_32_bits():
    rows, width = 600000, 4096
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    tail, weight, bias, grad = inputs(100, width, torch.bfloat16, torch.bfloat16)
    x[-100:] = tail
    out, mean, rstd = st.layer_norm(x, weight, bias)
    forward_matches((out[-100:], mean[-100:], rstd[-100:]), tail, weight, bias, 1e-5)
    assert torch.equal(out[:1000], bias.expand(1000, width))
    all_grad = torch.zeros_like(x)
    all_grad[-100:] = grad
    got = st.layer_norm_backward(all_grad, x, weight, mean, rstd)
    for value, (want, bound) in zip((got[0][-100:], got[1], got[2]), gradients(grad, tail, weight, 1e-5)):
        ref.within(value, want.cpu().numpy(), (bound + ref.rounded(value.dtype, want.abs())).cpu().numpy())

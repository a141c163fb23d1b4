"""A sparse expert layer put together from the operators, as a program runs
it: layer norm, routing limited to groups, tokens sorted by expert, the experts'
products and back, with every gradient; and in 8 bits for inference."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref

pytestmark = pytest.mark.gpu
TOKENS, WIDTH, HIDDEN, EXPERTS, K = 300, 256, 384, 16, 3
ROUTING = dict(num_groups=4, groups_kept=2)


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def parameters(dtype):
    return dict(weight=(1 + 0.1 * randn(WIDTH, seed=1)).to(dtype), bias=0.1 * randn(WIDTH, seed=2, dtype=dtype),
                router=randn(WIDTH, EXPERTS, seed=3, dtype=dtype) * WIDTH ** -0.5,
                up=randn(EXPERTS, HIDDEN, WIDTH, seed=4, dtype=dtype) * WIDTH ** -0.5,
                down=randn(EXPERTS, WIDTH, HIDDEN, seed=5, dtype=dtype) * HIDDEN ** -0.5)


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        out, mean, rstd = st.layer_norm(x, weight, bias)
        ctx.save_for_backward(x, weight, mean, rstd)
        return out

    @staticmethod
    def backward(ctx, grad):
        return st.layer_norm_backward(grad, *ctx.saved_tensors)


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits):
        ids, weights = st.route(logits, K, **ROUTING)
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    def backward(ctx, _, grad):
        return st.route_backward(grad, *ctx.saved_tensors)


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, groups):
        ctx.groups = groups
        return st.dispatch(x, groups)

    @staticmethod
    def backward(ctx, grad):
        return st.dispatch_backward(grad, ctx.groups), None


class Product(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, groups):
        ctx.save_for_backward(rows, weights)
        ctx.groups = groups
        return st.expert_matmul(rows, weights, groups)

    @staticmethod
    def backward(ctx, grad):
        return *st.expert_matmul_backward(grad, *ctx.saved_tensors, ctx.groups), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, groups):
        ctx.save_for_backward(rows, weights)
        ctx.groups = groups
        return st.combine(rows, groups, weights)

    @staticmethod
    def backward(ctx, grad):
        rows, weights = ctx.saved_tensors
        return *st.combine_backward(grad, rows, ctx.groups, weights), None


def layer(x, p):
    h = Norm.apply(x, p["weight"], p["bias"])
    ids, weights = Route.apply((h @ p["router"]).float())
    groups = st.group_by_expert(ids, EXPERTS)
    rows = Product.apply(torch.relu(Product.apply(Dispatch.apply(h, groups), p["up"], groups)), p["down"], groups)
    return x + Combine.apply(rows, weights, groups), ids


def plain(x, p, ids):
    """The same in 64 bits by torch, with the choice of experts given."""
    h = torch.nn.functional.layer_norm(x, (WIDTH,), p["weight"], p["bias"])
    scores = torch.softmax(h @ p["router"], 1).gather(1, ids.long())
    scores = scores / scores.sum(1, keepdim=True)
    hidden = torch.relu(torch.einsum("td,tkhd->tkh", h, p["up"][ids.long()]))
    return x + torch.einsum("tkh,tkdh,tk->td", hidden, p["down"][ids.long()], scores)


def apart(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_training_step(dtype):
    # Seven results in 16 bits lie between x and out, and as many on the way back, each off by at most u = eps / 2 of
    # its value: 14 u in all to first order, were the sums' terms of one sign. They are not: a sum of n terms of either
    # sign is about n^(1/2) times smaller than their magnitudes, while the terms' roundings, which are independent,
    # grow by n^(1/2) too; so relative to norms each stage adds at most its own u. The norm's gradient takes out two
    # means, which leaves at least half of what it gets here: a factor of 2, and one for relu's and the weights' own.
    p = {name: value.requires_grad_() for name, value in parameters(dtype).items()}
    x = randn(TOKENS, WIDTH, seed=6, dtype=dtype).requires_grad_()
    out, ids = layer(x, p)
    grad = randn(TOKENS, WIDTH, seed=7, dtype=dtype)
    out.backward(grad)
    p64 = {name: value.detach().double().requires_grad_() for name, value in p.items()}
    x64 = x.detach().double().requires_grad_()
    want = plain(x64, p64, ids)
    want.backward(grad.double())
    bound = 14 * 4 * torch.finfo(dtype).eps / 2
    assert apart(out.detach(), want.detach()) <= bound and apart(x.grad, x64.grad) <= bound
    for name in p:
        assert apart(p[name].grad, p64[name].grad) <= bound, name


def quantized(w):
    """[experts, out, width] in 8 bits with a scale for each 128 by 128 values (all sizes are multiples of 128)."""
    e, n, k = w.shape
    tiles = w.float().reshape(e, n // 128, 128, k // 128, 128)
    most = tiles.abs().amax((2, 4), keepdim=True)
    return (tiles * (448 / most)).to(torch.float8_e4m3fn).reshape(e, n, k), (most / 448).reshape(e, n // 128, k // 128)


def test_inference_in_8_bits_captured():
    p = parameters(torch.bfloat16)
    up, up_scales = quantized(p["up"])
    down, down_scales = quantized(p["down"])
    x = randn(TOKENS, WIDTH, seed=6, dtype=torch.bfloat16)

    def run():
        h, _, _ = st.layer_norm(x, p["weight"], p["bias"])
        ids, weights = st.route((h @ p["router"]).float(), K, **ROUTING)
        groups = st.group_by_expert(ids, EXPERTS)
        values, scales = st.quantize_rows(h)  # each token once, then its bytes to its experts
        rows = st.expert_matmul(st.dispatch(values, groups), up, groups, row_scales=st.dispatch(scales, groups),
                                weight_scales=up_scales)
        values, scales = st.quantize_rows(torch.relu(rows))
        rows = st.expert_matmul(values, down, groups, row_scales=scales, weight_scales=down_scales)
        return x + st.combine(rows, groups, weights), ids

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, ids = run()
    for seed in (6, 8):
        x.copy_(randn(TOKENS, WIDTH, seed=seed, dtype=torch.bfloat16))
        graph.replay()
        eager, eager_ids = run()
        assert torch.equal(out, eager) and torch.equal(ids, eager_ids)
        # against the weights that the 8 bits stand for: what is left are two quantised inputs (2^-4 of a value at
        # most, and 448's share of a block), and roundings to 16 bits, which are far below
        p64 = {name: value.double() for name, value in p.items()}
        for name, values, scales in (("up", up, up_scales), ("down", down, down_scales)):
            p64[name] = values.double() * scales.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        want = plain(x.double(), p64, ids) - x.double()
        assert apart(out.double() - x.double(), want) <= 2 * 2.0 ** -4 + 16 * 2.0 ** -8
    assert st.read_device_error() == 0


def test_tokens_with_no_expert_and_unused_experts():
    p = parameters(torch.bfloat16)
    x = randn(40, WIDTH, seed=6, dtype=torch.bfloat16)
    logits = randn(40, EXPERTS, seed=8)
    logits[:, 8:] = -float("inf")
    logits[::5] = -float("inf")
    ids, weights = st.route(logits, K, **ROUTING)
    assert (ids[::5] == -1).all()
    groups = st.group_by_expert(ids, EXPERTS)
    rows = st.dispatch(x, groups)
    out = st.expert_matmul(rows, p["up"], groups)
    grad_rows, grad_up = st.expert_matmul_backward(out, rows, p["up"], groups)
    kept = int(groups.offsets[-1])
    assert kept <= 32 * K and not out[kept:].any() and not grad_rows[kept:].any() and not grad_up[8:].any()
    back = st.combine(out, groups, weights)
    assert not back[::5].any() and back[1].any()

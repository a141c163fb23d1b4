"""The experts' products against their definition in 64 bits.

Where rows and weights are small whole numbers every product and sum is exact
in 32 bits (below 2^24), so results in float32 have to be equal. Otherwise a
sum of n terms, added in 32 bits by cutting off or rounding, is off by at most
(n + 1) 2^-23 times the sum of the terms' magnitudes, and its last rounding
follows."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref
from tests.test_gpu_rows_experts import ids_of

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
SHAPES = [  # tokens, k, experts, width, out, dropped
    (1, 1, 1, 8, 8, 0), (1, 8, 64, 128, 128, 0), (3, 2, 4, 64, 24, 0), (7, 3, 5, 72, 40, 0.3), (33, 1, 1, 200, 256, 0),
    (100, 6, 60, 1000, 1096, 0.1), (300, 2, 3, 256, 264, 0), (1500, 1, 1, 64, 520, 0), (700, 3, 2, 136, 136, 0.2),
    (2731, 3, 7, 136, 8, 0.1), (257, 1, 1, 320, 384, 0), (50, 2, 8, 128, 128, 1.0), (90, 4, 200, 64, 72, 0)]


def whole(*shape, seed, dtype, most=3):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).to(torch.float32).to(dtype).cuda()


def randn(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def groups_of(tokens, k, experts, dropped, seed=0):
    return st.group_by_expert(ids_of(tokens, k, experts, seed, dropped).cuda(), experts)


def by_expert(groups, call):
    """call(expert, rows of it) for every expert with rows."""
    bounds = groups.offsets.tolist()
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if b > a:
            call(e, slice(a, b))


def product(rows, weights, groups):
    """rows and weights in 64 bits: the product and the sum of its terms' magnitudes."""
    out = torch.zeros(rows.shape[0], weights.shape[1], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)

    def one(e, at):
        out[at] = rows[at] @ weights[e].t()
        size[at] = rows[at].abs() @ weights[e].abs().t()
    by_expert(groups, one)
    return out, size


def weights_gradient(grad, rows, weights, groups):
    out, size = torch.zeros_like(weights), torch.zeros_like(weights)

    def one(e, at):
        out[e] = grad[at].t() @ rows[at]
        size[e] = grad[at].abs().t() @ rows[at].abs()
    by_expert(groups, one)
    return out, size


def near(got, want, size, terms):
    bound = (terms + 1) * 2.0 ** -23 * size + ref.rounded(got.dtype, want.abs())
    ref.within(got, want.cpu().numpy(), bound.cpu().numpy())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,k,experts,width,out,dropped", SHAPES)
def test_products_and_gradients_of_whole_numbers(tokens, k, experts, width, out, dropped, dtype):
    groups = groups_of(tokens, k, experts, dropped)
    n = tokens * k
    rows = whole(n, width, seed=1, dtype=dtype)
    weights = whole(experts, out, width, seed=2, dtype=dtype)
    grad = whole(n, out, seed=3, dtype=dtype)
    kept = int(groups.offsets[-1])
    # what no expert has is not read into anything
    rows[kept:] = float("nan")
    grad[kept:] = float("inf")
    want, _ = product(rows.double(), weights.double(), groups)
    for type in (torch.float32, dtype):
        got = st.expert_matmul(rows, weights, groups, out_dtype=type)
        assert got.dtype == type and torch.equal(got, want.to(type))
    grad_rows, grad_weights = st.expert_matmul_backward(grad, rows, weights, groups, dtype=torch.float32)
    assert torch.equal(grad_rows, product(grad.double(), weights.double().transpose(1, 2), groups)[0].to(dtype))
    want, _ = weights_gradient(grad.double(), rows.double(), weights.double(), groups)
    assert torch.equal(grad_weights, want.float())
    assert torch.equal(st.expert_matmul_backward(grad, rows, weights, groups)[1], want.to(dtype))


@pytest.mark.parametrize("tokens,k,experts,width,out,dropped", SHAPES)
def test_weights_in_the_other_layout(tokens, k, experts, width, out, dropped):
    # [experts, width, out] in memory; the gradient comes in that layout too
    groups = groups_of(tokens, k, experts, dropped)
    rows = whole(tokens * k, width, seed=1, dtype=torch.bfloat16)
    weights = whole(experts, width, out, seed=2, dtype=torch.bfloat16).transpose(1, 2)
    grad = whole(tokens * k, out, seed=3, dtype=torch.bfloat16)
    got = st.expert_matmul(rows, weights, groups, out_dtype=torch.float32)
    assert torch.equal(got, product(rows.double(), weights.double(), groups)[0].float())
    grad_rows, grad_weights = st.expert_matmul_backward(grad, rows, weights, groups)
    plain = st.expert_matmul_backward(grad, rows, weights.contiguous(), groups)
    assert torch.equal(grad_rows, plain[0]) and torch.equal(grad_weights, plain[1])
    assert grad_weights.transpose(1, 2).is_contiguous()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,k,experts,width,out,dropped", SHAPES[5:9])
def test_products_and_gradients(tokens, k, experts, width, out, dropped, dtype):
    groups = groups_of(tokens, k, experts, dropped)
    rows, grad = randn(tokens * k, width, seed=1, dtype=dtype), randn(tokens * k, out, seed=2, dtype=dtype)
    weights = randn(experts, out, width, seed=3, dtype=dtype)
    x, w, g = rows.double(), weights.double(), grad.double()
    near(st.expert_matmul(rows, weights, groups), *product(x, w, groups), width)
    near(st.expert_matmul(rows, weights, groups, out_dtype=torch.float32), *product(x, w, groups), width)
    grad_rows, grad_weights = st.expert_matmul_backward(grad, rows, weights, groups)
    near(grad_rows, *product(g, w.transpose(1, 2), groups), out)
    near(grad_weights, *weights_gradient(g, x, w, groups), tokens * k)
    # along a direction: the product is linear in each, so differences are the formula itself
    dx = randn(tokens * k, width, seed=4, dtype=dtype).double()
    ahead = (g * (product(x + dx, w, groups)[0] - product(x - dx, w, groups)[0])).sum() / 2
    bound = ((out + 1) * 2.0 ** -23 * product(g, w.transpose(1, 2), groups)[1] + ref.rounded(dtype, grad_rows.double().abs()) * 1.01)
    assert abs(float((grad_rows.double() * dx).sum() - ahead)) <= float((bound * dx.abs()).sum()) * 1.01


@pytest.mark.parametrize("out", [1, 7, 129, 1001])
def test_any_number_of_outputs(out):
    groups = groups_of(150, 2, 5, 0.1)
    rows, weights = whole(300, 136, seed=1, dtype=torch.bfloat16), whole(5, out, 136, seed=2, dtype=torch.bfloat16)
    want = product(rows.double(), weights.double(), groups)[0]
    for type in (torch.float32, torch.bfloat16, torch.float16):
        assert torch.equal(st.expert_matmul(rows, weights, groups, out_dtype=type), want.to(type))
    # a result that does not start on 16 bytes, and what lies around it
    around = torch.full((300 * 64 + 2,), 7.0, device="cuda", dtype=torch.bfloat16)
    weights = whole(5, 64, 136, seed=3, dtype=torch.bfloat16)
    st.expert_matmul(rows, weights, groups, out=around[1:-1].view(300, 64))
    assert torch.equal(around[1:-1].view(300, 64), product(rows.double(), weights.double(), groups)[0].bfloat16())
    assert around[0] == around[-1] == 7


F8_SHAPES = [  # tokens, k, experts, width, out, dropped
    (1, 1, 1, 16, 1, 0), (1, 8, 64, 128, 128, 0), (3, 2, 4, 128, 129, 0), (7, 3, 5, 144, 40, 0.3), (100, 6, 60, 1040, 1000, 0.1),
    (300, 2, 3, 256, 1001, 0), (1500, 1, 1, 640, 520, 0), (9000, 1, 3, 272, 392, 0.1), (50, 2, 8, 128, 128, 1.0),
    (2000, 4, 16, 2048, 640, 0), (129, 1, 1, 512, 16, 0), (40000, 1, 2, 128, 264, 0)]


def eight_bits(tokens, k, experts, width, out, exact):
    """Rows, weights and scales; with `exact`, whole numbers and powers of two."""
    blocks, out_blocks = -(-width // 128), -(-out // 128)
    if exact:
        power = lambda *shape, seed: torch.exp2(whole(*shape, seed=seed, dtype=torch.float32, most=2))
        return (whole(tokens * k, width, seed=1, dtype=F8), whole(experts, out, width, seed=2, dtype=F8),
                power(tokens * k, blocks, seed=3), power(experts, out_blocks, blocks, seed=4))
    scale = lambda *shape, seed: 0.01 * torch.exp(randn(*shape, seed=seed, dtype=torch.float32))
    return (randn(tokens * k, width, seed=1, dtype=torch.float32).mul(50).to(F8),
            randn(experts, out, width, seed=2, dtype=torch.float32).mul(50).to(F8),
            scale(tokens * k, blocks, seed=3), scale(experts, out_blocks, blocks, seed=4))


def spread(scales, rows, n, width):
    return scales.double().repeat_interleave(rows, -2)[..., :n, :].repeat_interleave(128, -1)[..., :width]


def product8(rows, weights, row_scales, weight_scales, groups):
    x = rows.double() * spread(row_scales, 1, *rows.shape)
    w = weights.double() * spread(weight_scales, 128, *weights.shape[1:])
    return product(x, w, groups)


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("tokens,k,experts,width,out,dropped", F8_SHAPES)
def test_products_in_8_bits(tokens, k, experts, width, out, dropped, exact):
    groups = groups_of(tokens, k, experts, dropped)
    rows, weights, row_scales, weight_scales = eight_bits(tokens, k, experts, width, out, exact)
    kept = int(groups.offsets[-1])
    rows.view(torch.uint8)[kept:] = 0x7f  # NaN
    row_scales[kept:] = float("nan")
    want, size = product8(rows, weights, row_scales, weight_scales, groups)
    for type in (torch.float32, torch.bfloat16, torch.float16):
        got = st.expert_matmul(rows, weights, groups, row_scales=row_scales, weight_scales=weight_scales, out_dtype=type)
        assert got.dtype == type
        if exact:
            # at most 2048 terms of 9 2^4, all multiples of 2^-4: sums below 2^24 times that
            assert torch.equal(got, want.to(type))
        else:
            # beside the sum's additions each block's is scaled: three roundings more
            near(got, want, size, width + 3)
    if not exact:
        assert st.expert_matmul(rows, weights, groups, row_scales=row_scales,
                                weight_scales=weight_scales).dtype == torch.bfloat16


@pytest.mark.parametrize("eight", [False, True])
def test_a_row_alone_is_touched_by_its_own_values(eight):
    # NaN and infinities in one row, or one expert's weights, stay there
    groups = groups_of(400, 2, 3, 0.0)
    bounds = groups.offsets.tolist()
    width, out = 272, 200
    if eight:
        rows, weights, rs, ws = eight_bits(400, 2, 3, width, out, True)
        how = dict(row_scales=rs, weight_scales=ws)
    else:
        rows, weights = whole(800, width, seed=1, dtype=torch.bfloat16), whole(3, out, width, seed=2, dtype=torch.bfloat16)
        how = {}
    clean = st.expert_matmul(rows, weights, groups, **how)
    bad_row = bounds[1] + 5
    rows.view(torch.uint8 if eight else torch.int16)[bad_row, width - 1] = 0x7f if eight else 0x7fc0
    weights.view(torch.uint8 if eight else torch.int16)[0, 3] = 0x7f if eight else 0x7fc0
    got = st.expert_matmul(rows, weights, groups, **how)
    nan = torch.zeros_like(clean, dtype=torch.bool)
    nan[bad_row] = True
    nan[:bounds[1], 3] = True
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], clean[~nan])
    if not eight:
        weights[0] = float("nan")
        grad = whole(800, out, seed=3, dtype=torch.bfloat16)
        grad_rows, grad_weights = st.expert_matmul_backward(grad, rows, weights, groups)
        assert torch.isnan(grad_rows[:bounds[1]]).all() and torch.isfinite(grad_rows[bounds[1]:]).all()
        assert torch.isfinite(grad_weights[0]).all() and torch.isfinite(grad_weights[2]).all()
        assert torch.isnan(grad_weights[1, :, width - 1]).all() and torch.isfinite(grad_weights[1, :, :width - 1]).all()


def test_layouts():
    # parts of wider tensors, one row for all, odd starts, experts some distance apart
    groups = groups_of(60, 3, 4, 0.1)
    n, width, out = 180, 64, 40
    wide = whole(n, 200, seed=1, dtype=torch.bfloat16)
    weights = whole(4, out, width, seed=2, dtype=torch.bfloat16)
    far = whole(4 * (out * width + 24) + 8, seed=3, dtype=torch.bfloat16)
    apart = far.as_strided((4, out, width), (out * width + 24, width, 1))
    odd = far[1:].as_strided((4, out, width), (out * width + 24, width, 1))
    one = weights[:1].expand(4, out, width)
    # 16 bits: rows at 16-byte steps (read in place), at others (copied), and one row for all (copied)
    for rows in (wide[:, 8:72], wide[:, 5:69], wide[:1, :64].expand(n, 64), wide.t().contiguous().t()[:, :64]):
        for w in (weights, apart, odd, one, weights[:, :, :].flip(0)):
            want = product(rows.double(), w.double(), groups)[0]
            assert torch.equal(st.expert_matmul(rows, w, groups, out_dtype=torch.float32), want.float())
        grad = wide[:, 100:100 + out]
        got = st.expert_matmul_backward(grad, rows, apart, groups, dtype=torch.float32)
        assert torch.equal(got[0], product(grad.double(), apart.double().transpose(1, 2), groups)[0].bfloat16())
        assert torch.equal(got[1], weights_gradient(grad.double(), rows.double(), apart.double(), groups)[0].float())
    # 8 bits: the same, and scales in a wider tensor and one for all
    rows, w8, rs, ws = eight_bits(60, 3, 4, 144, 40, True)
    broad = torch.zeros(n, 200, device="cuda").to(F8)
    for at in (16, 7):
        part = broad[:, at:at + 144]
        part.view(torch.uint8).copy_(rows.view(torch.uint8))
        scales = torch.cat([rs, rs], 1)[:, 1:3]
        want = product8(part, w8, scales, ws, groups)[0]
        got = st.expert_matmul(part, w8, groups, row_scales=scales, weight_scales=ws, out_dtype=torch.float32)
        assert torch.equal(got, want.float())
    turned = w8.transpose(1, 2).contiguous().transpose(1, 2)
    got = st.expert_matmul(rows, turned, groups, row_scales=rs[:1].expand_as(rs), weight_scales=ws, out_dtype=torch.float32)
    assert torch.equal(got, product8(rows, w8, rs[:1].expand_as(rs), ws, groups)[0].float())


def test_results_repeat_and_calls_run_together():
    groups = groups_of(900, 4, 20, 0.1)
    rows, weights = randn(3600, 512, seed=1, dtype=torch.bfloat16), randn(20, 384, 512, seed=2, dtype=torch.bfloat16)
    grad = randn(3600, 384, seed=3, dtype=torch.bfloat16)
    first = (st.expert_matmul(rows, weights, groups), *st.expert_matmul_backward(grad, rows, weights, groups))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            got.append((st.expert_matmul(rows, weights, groups, stream=s),
                        *st.expert_matmul_backward(grad, rows, weights, groups, stream=s)))
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(a, b) for a, b in zip(one, first))
    assert st.read_device_error() == 0


def test_graph():
    groups = groups_of(300, 2, 6, 0.1)
    rows, weights = whole(600, 256, seed=1, dtype=torch.bfloat16), whole(6, 128, 256, seed=2, dtype=torch.bfloat16)
    grad = whole(600, 128, seed=3, dtype=torch.bfloat16)
    ids = ids_of(300, 2, 6, 0, 0.1).cuda()
    out = torch.empty(600, 128, device="cuda", dtype=torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = st.group_by_expert(ids, 6)
        st.expert_matmul(rows, weights, captured, out=out)
        grad_rows, grad_weights = st.expert_matmul_backward(grad, rows, weights, captured)
    for seed in (5, 6):
        # other rows and another grouping in the same memory
        rows.copy_(whole(600, 256, seed=seed, dtype=torch.bfloat16))
        ids.copy_(ids_of(300, 2, 6, seed, 0.2).cuda())
        graph.replay()
        groups = st.group_by_expert(ids, 6)
        assert torch.equal(out, product(rows.double(), weights.double(), groups)[0].bfloat16())
        assert torch.equal(grad_rows, product(grad.double(), weights.double().transpose(1, 2), groups)[0].bfloat16())
        assert torch.equal(grad_weights, weights_gradient(grad.double(), rows.double(), weights.double(), groups)[0].bfloat16())


def test_outputs_and_no_rows():
    groups = groups_of(10, 2, 4, 0.0)
    rows, weights = whole(20, 64, seed=1, dtype=torch.float16), whole(4, 32, 64, seed=2, dtype=torch.float16)
    out = torch.full((20, 32), 7.0, device="cuda", dtype=torch.float32)
    version = out._version
    assert st.expert_matmul(rows, weights, groups, out=out) is not None and out._version > version
    assert torch.equal(out, product(rows.double(), weights.double(), groups)[0].float())
    none = st.ExpertGroups(torch.zeros(5, dtype=torch.int64, device="cuda"),
                           torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert st.expert_matmul(rows[:0], weights, none).shape == (0, 32)
    grad_rows, grad_weights = st.expert_matmul_backward(rows[:0, :32], rows[:0], weights, none)
    assert grad_rows.shape == (0, 64) and not grad_weights.any()


def test_offsets_that_are_no_offsets_stay_in_bounds():
    # below an earlier one, negative, past the rows: taken as the nearest that are not
    rows, weights = whole(50, 64, seed=1, dtype=torch.bfloat16), whole(4, 32, 64, seed=2, dtype=torch.bfloat16)
    of = torch.tensor([-5, 30, 10, 2 ** 40, 20], dtype=torch.int64, device="cuda")
    as_taken = torch.tensor([0, 30, 30, 50, 50], dtype=torch.int64, device="cuda")
    some = groups_of(25, 2, 4, 0.0)
    got = st.expert_matmul(rows, weights, some._replace(offsets=of))
    assert torch.equal(got, st.expert_matmul(rows, weights, some._replace(offsets=as_taken)))
    assert torch.equal(got, product(rows.double(), weights.double(), some._replace(offsets=as_taken))[0].bfloat16())


def test_past_32_bits():
    # 600 000 rows of 4096: the last rows' offsets need 64 bits, in elements and in bytes
    n, width, out = 600000, 4096, 16
    ids = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    ids[-100:] = 1
    groups = st.group_by_expert(ids, 2)
    rows = torch.ones(n, width, dtype=torch.bfloat16, device="cuda")
    rows[-100:] = 2
    weights = whole(2, out, width, seed=2, dtype=torch.bfloat16)
    got = st.expert_matmul(rows, weights, groups, out_dtype=torch.float32)
    sums = weights.double().sum(2).float()
    assert torch.equal(got[:-100], sums[:1].expand(n - 100, out)) and torch.equal(got[-100:], 2 * sums[1:].expand(100, out))
    grad = torch.ones(n, out, dtype=torch.bfloat16, device="cuda")
    grad_rows, grad_weights = st.expert_matmul_backward(grad, rows, weights, groups, dtype=torch.float32)
    columns = weights.double().sum(1).bfloat16()
    assert torch.equal(grad_rows[-1], columns[1]) and torch.equal(grad_rows[0], columns[0])
    assert torch.equal(grad_weights[0], torch.full((out, width), n - 100.0, device="cuda"))
    assert torch.equal(grad_weights[1], torch.full((out, width), 200.0, device="cuda"))

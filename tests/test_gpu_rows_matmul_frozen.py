"""The rows' gradient of a frozen layer in 8 bits: the same product of the
quantised gradient with the weights, and their scales, transposed."""
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests.test_gpu_rows_matmul import by_expert, eight_bits, groups_of, near, randn, spread, whole, F8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("tokens,k,experts,width,out,dropped", [(1, 1, 1, 16, 16, 0), (7, 3, 5, 144, 48, 0.3), (100, 6, 60, 1040, 1008, 0.1),
                                                                (300, 2, 3, 256, 384, 0), (20000, 1, 2, 272, 528, 0.1)])
def test_gradient_of_the_rows(tokens, k, experts, width, out, dropped, exact):
    groups = groups_of(tokens, k, experts, dropped)
    n = tokens * k
    _, weights, _, weight_scales = eight_bits(tokens, k, experts, width, out, exact)
    if exact:
        # whole numbers and powers of two: sums of at most 1008 terms of 9 2^4 in steps of 2^-4, all exact
        values = whole(n, out, seed=7, dtype=F8)
        scales = torch.exp2(whole(n, -(-out // 128), seed=8, dtype=torch.float32, most=2))
    else:
        values, scales = st.quantize_rows(randn(n, out, seed=7, dtype=torch.bfloat16))
    g = values.double() * spread(scales, 1, n, out)
    w = weights.double() * spread(weight_scales, 128, out, width)
    want, size = (torch.zeros(n, width, dtype=torch.float64, device="cuda") for _ in range(2))

    def one(e, at):
        want[at] = torch.einsum("rn,nk->rk", g[at], w[e])
        size[at] = torch.einsum("rn,nk->rk", g[at].abs(), w[e].abs())
    by_expert(groups, one)
    laid_out = weights.transpose(1, 2).contiguous(), weight_scales.transpose(1, 2).contiguous()
    for w8, ws in (laid_out, (weights.transpose(1, 2), weight_scales.transpose(1, 2))):
        for type in (torch.float32, torch.bfloat16):
            got = st.expert_matmul(values, w8, groups, row_scales=scales, weight_scales=ws, out_dtype=type)
            assert got.shape == (n, width) and got.dtype == type
            if exact:
                assert torch.equal(got, want.to(type))
            else:
                near(got, want, size, out + 3)  # each block's sum is scaled: three roundings beside the additions

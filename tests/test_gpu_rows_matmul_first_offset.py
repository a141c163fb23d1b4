"""The experts' products where the first offset is above 0: the rows before it
belong to no expert, like those behind the last one. They are read into
nothing, and their rows of the result are zeros."""
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests.test_gpu_rows_matmul import eight_bits, product, product8, weights_gradient, whole

pytestmark = pytest.mark.gpu


def starting_at(first, counts, behind):
    bounds = torch.cumsum(torch.tensor([first, *counts]), 0)
    n = int(bounds[-1]) + behind
    groups = st.ExpertGroups(bounds.cuda(), torch.zeros(n, 1, dtype=torch.int32, device="cuda"),
                             torch.zeros(n, dtype=torch.int32, device="cuda"))
    return groups, n, torch.cat([torch.arange(first), torch.arange(n - behind, n)]).cuda()


CASES = [(1, [3, 0, 5], 0, 64, 72), (137, [300, 0, 40, 129], 5, 144, 264), (5, [0, 0], 0, 64, 8), (40, [7], 3, 1040, 1000),
         (2, [64, 64], 0, 128, 129)]


@pytest.mark.parametrize("first,counts,behind,width,out", CASES)
def test_16_bits(first, counts, behind, width, out):
    groups, n, nobody = starting_at(first, counts, behind)
    experts = len(counts)
    rows, weights = whole(n, width, seed=1, dtype=torch.bfloat16), whole(experts, out, width, seed=2, dtype=torch.bfloat16)
    rows[nobody] = float("nan")
    want = product(rows.double(), weights.double(), groups)[0]
    assert not want[nobody].any()
    for type in (torch.float32, torch.bfloat16):
        got = torch.full((n, out), 7.0, device="cuda", dtype=type)
        st.expert_matmul(rows, weights, groups, out=got)
        assert torch.equal(got, want.to(type))
    if out % 8:
        return
    turned = weights.transpose(1, 2).contiguous().transpose(1, 2)
    got = torch.full((n, out), 7.0, device="cuda", dtype=torch.float32)
    assert torch.equal(st.expert_matmul(rows, turned, groups, out=got), want.float())
    grad = whole(n, out, seed=3, dtype=torch.bfloat16)
    grad[nobody] = float("inf")
    # memory of the results' size that holds something else
    for shape in ((n, width), (experts, out, width)):
        torch.full(shape, 7.0, device="cuda", dtype=torch.bfloat16)
    grad_rows, grad_weights = st.expert_matmul_backward(grad, rows, weights, groups)
    assert torch.equal(grad_rows, product(grad.double(), weights.double().transpose(1, 2), groups)[0].bfloat16())
    assert torch.equal(grad_weights, weights_gradient(grad.double(), rows.double(), weights.double(), groups)[0].bfloat16())


@pytest.mark.parametrize("first,counts,behind,width,out", CASES + [(137, [20000, 19000], 50, 128, 264)])  # the last by pairs
def test_8_bits(first, counts, behind, width, out):
    groups, n, nobody = starting_at(first, counts, behind)
    rows, weights, rs, ws = eight_bits(n, 1, len(counts), width, out, True)
    rows.view(torch.uint8)[nobody] = 0x7f  # NaN
    rs[nobody] = float("nan")
    want = product8(rows, weights, rs, ws, groups)[0]
    for type in (torch.float32, torch.bfloat16):
        got = torch.full((n, out), 7.0, device="cuda", dtype=type)
        st.expert_matmul(rows, weights, groups, row_scales=rs, weight_scales=ws, out=got)
        assert torch.equal(got, want.to(type))


def test_all_rows_before_the_first_offset():
    groups, n, _ = starting_at(50, [0, 0, 0], 0)
    rows, weights = whole(n, 64, seed=1, dtype=torch.bfloat16), whole(3, 32, 64, seed=2, dtype=torch.bfloat16)
    past = groups._replace(offsets=groups.offsets + 1000)  # past the rows: the same
    for of in (groups, past):
        got = torch.full((n, 32), 7.0, device="cuda", dtype=torch.bfloat16)
        assert not st.expert_matmul(rows, weights, of, out=got).any()

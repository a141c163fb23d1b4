"""The experts' products with as many experts as their tiles' search has borders
at, with experts that all have other numbers of rows, and one call after the
other on a stream."""
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests.test_gpu_rows_matmul import eight_bits, product, product8, weights_gradient, whole

pytestmark = pytest.mark.gpu


def groups_with(counts, dropped=0):
    """Expert e has counts[e] rows; `dropped` slots have none."""
    ids = torch.cat([torch.full((n,), e, dtype=torch.int32) for e, n in enumerate(counts)] +
                    [torch.full((dropped,), -1, dtype=torch.int32)])
    order = torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))
    groups = st.group_by_expert(ids[order].view(-1, 1).cuda(), len(counts))
    assert (groups.offsets[1:] - groups.offsets[:-1]).tolist() == list(counts)
    return groups, len(ids)


def check(groups, n, experts, width, out):
    rows, weights = whole(n, width, seed=1, dtype=torch.bfloat16), whole(experts, out, width, seed=2, dtype=torch.bfloat16)
    grad = whole(n, out, seed=3, dtype=torch.bfloat16)
    got = st.expert_matmul(rows, weights, groups, out_dtype=torch.float32)
    assert torch.equal(got, product(rows.double(), weights.double(), groups)[0].float())
    grad_rows, grad_weights = st.expert_matmul_backward(grad, rows, weights, groups, dtype=torch.float32)
    assert torch.equal(grad_rows, product(grad.double(), weights.double().transpose(1, 2), groups)[0].bfloat16())
    assert torch.equal(grad_weights, weights_gradient(grad.double(), rows.double(), weights.double(), groups)[0].float())
    rows, weights, rs, ws = eight_bits(n, 1, experts, width, out, True)
    got = st.expert_matmul(rows, weights, groups, row_scales=rs, weight_scales=ws, out_dtype=torch.float32)
    assert torch.equal(got, product8(rows, weights, rs, ws, groups)[0].float())


@pytest.mark.parametrize("experts", [1, 2, 31, 32, 33, 63, 64, 65, 383, 384, 385, 992, 993, 1023, 1024])
def test_numbers_of_experts(experts):
    counts = [(7 * e) % 5 if experts > 2 else 40 for e in range(experts)]
    groups, n = groups_with(counts, dropped=11)
    check(groups, n, experts, 64, 72)


@pytest.mark.parametrize("first", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 769, 1025])
def test_numbers_of_rows(first):
    # widths of tiles, and an expert's last block of rows, at their borders; experts without rows between them
    groups, n = groups_with([first, 0, first + 1, 64, 0, 2 * first, 3], dropped=5)
    check(groups, n, 7, 144, 264)


@pytest.mark.parametrize("width,out", [(16, 8), (128, 8), (64, 128), (128, 136), (192, 248), (256, 256), (320, 512), (1024, 520)])
def test_sizes_of_weights(width, out):
    groups, n = groups_with([300, 40, 0, 130], dropped=3)
    check(groups, n, 4, width, out)


def test_one_call_after_the_other():
    # each starts while the one before it ends
    a, na = groups_with([300, 5, 0, 260])
    b, nb = groups_with([3] * 40)
    x, w = whole(na, 256, seed=1, dtype=torch.bfloat16), whole(4, 256, 256, seed=2, dtype=torch.bfloat16, most=1)
    y, v = whole(nb, 128, seed=3, dtype=torch.float16), whole(40, 64, 128, seed=4, dtype=torch.float16)
    r8, w8, rs, ws = eight_bits(na, 1, 4, 256, 200, True)
    weight = torch.ones(256, device="cuda")
    want = (product(x.double(), w.double(), a)[0].float(), product(y.double(), v.double(), b)[0].float(),
            product8(r8, w8, rs, ws, a)[0].float())
    norm = st.layer_norm(want[0], weight)[0]
    quantized = st.quantize_rows(want[0])
    torch.cuda.synchronize()
    for _ in range(20):
        one = st.expert_matmul(x, w, a, out_dtype=torch.float32)
        after = st.layer_norm(one, weight)[0]
        values, scales = st.quantize_rows(one)
        two = st.expert_matmul(y, v, b, out_dtype=torch.float32)
        three = st.expert_matmul(r8, w8, a, row_scales=rs, weight_scales=ws, out_dtype=torch.float32)
        for got, right in ((one, want[0]), (two, want[1]), (three, want[2]), (after, norm), (scales, quantized[1])):
            assert torch.equal(got, right)
        assert torch.equal(values.view(torch.uint8), quantized[0].view(torch.uint8))

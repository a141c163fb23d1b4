"""The weights' gradient where every tile ends inside a block of rows, next to
the rows of others: those hold NaN or very large values, and none of them may
reach a result, however often it is computed."""
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests.test_gpu_rows_matmul import weights_gradient, whole
from tests.test_gpu_rows_matmul_experts import groups_with

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [list(range(1, 64)), [65, 1, 127, 63] * 12, [1] * 200])
def test_rows_of_others_are_gone_before_the_products(counts):
    groups, n = groups_with(counts, dropped=9)
    width, out = 520, 264  # two tiles of each, the second ones in part
    rows, grad = whole(n, width, seed=1, dtype=torch.bfloat16), whole(n, out, seed=2, dtype=torch.bfloat16)
    weights = torch.empty(len(counts), out, width, dtype=torch.bfloat16, device="cuda")
    kept = int(groups.offsets[-1])
    # every second expert's rows are 2^40 times as large: a row taken for a neighbour's is seen there
    large = torch.zeros(n, 1, dtype=torch.bool, device="cuda")
    bounds = groups.offsets.tolist()
    for e in range(0, len(counts), 2):
        large[bounds[e]:bounds[e + 1]] = True
    rows = torch.where(large, rows * 2.0 ** 40, rows)
    rows[kept:] = float("nan")
    grad[kept:] = float("nan")
    want = weights_gradient(grad.double(), rows.double(), weights.double(), groups)[0].float()
    got = [st.expert_matmul_backward(grad, rows, weights.zero_(), groups, dtype=torch.float32)[1] for _ in range(30)]
    assert all(torch.equal(g, want) for g in got)
    assert st.read_device_error() == 0

"""Rows wider than a group of threads takes at a time, on odd widths too, and
the widest that a sum is given."""
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import test_gpu_rows_experts as experts

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,k,num_experts,width,dropped", [
    (33, 3, 9, 1025, 0.2), (9, 2, 8, 2047, 0), (300, 4, 16, 2047, 0.1), (40, 9, 12, 5001, 0.1), (7, 17, 20, 1023, 0.3)])
def test_several_steps_of_odd_rows(tokens, k, num_experts, width, dropped, dtype):
    experts.test_there_and_back(tokens, k, num_experts, width, dropped, dtype)


def test_more_tiles_of_columns_than_a_grid_has():
    # a group of threads takes 1024 columns of 32 bits, and a grid has 65535
    # groups beside one another; powers of two, so that products are exact
    width = 65535 * 1024 + 4
    row = torch.randn(1, width, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    rows = row.expand(8, width)
    groups = st.group_by_expert(torch.zeros(8, 1, dtype=torch.int32, device="cuda"), 1)
    weights = 2.0 ** torch.arange(-4, 4, device="cuda").float()[:, None]
    out = st.combine(rows, groups, weights)
    for t in range(8):
        assert torch.equal(out[t], row[0] * weights[t])
    del out
    out = st.dispatch_backward(rows, groups)
    assert all(torch.equal(out[t], row[0]) for t in range(8))

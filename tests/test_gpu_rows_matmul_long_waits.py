"""The bound of a wait in the weights' gradient holds for a wait without
progress, not for an expert's rows: in the instrumented build the bound is a
fraction of what one expert's rows take, and the result is right all the
same."""
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests.test_gpu_rows_bounded_wait import BF16, DEFAULT_WAIT, F32, instr  # noqa: F401 (a fixture)
from tests.test_gpu_rows_matmul import whole

pytestmark = pytest.mark.gpu
# 0.5 ms; a block of 64 rows takes 64 cycles of the tensor cores at least, so 2^21 rows are 2^21 cycles or more
LIMIT, ROWS = 1 << 20, 1 << 21


@pytest.mark.parametrize("last", [0, 5])  # rows of nobody behind those of the last block
def test_rows_that_take_longer_than_the_bound(instr, last):  # noqa: F811
    a, b = whole(ROWS, 64, seed=1, dtype=torch.bfloat16, most=1), whole(ROWS, 128, seed=2, dtype=torch.bfloat16, most=1)
    if last:
        a[-last:] = float("nan")
    offsets = torch.tensor([0, 0, ROWS - last], device="cuda")
    want = a[:ROWS - last].double().t() @ b[:ROWS - last].double()
    got = torch.full((2, 64, 128), 7.0, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    st.set_test_hooks(LIMIT, 0)
    try:
        status = instr.segtopk_expert_matmul_weights(BF16, a.data_ptr(), 64, 64, b.data_ptr(), 128, 128, ROWS, 2,
                                                     offsets.data_ptr(), F32, got.data_ptr(), stream)
        err = st.read_device_error(lib=instr)
    finally:
        st.set_test_hooks(DEFAULT_WAIT, 0)
    assert status == 0 and err == 0
    assert not got[0].any() and torch.equal(got[1], want.float())

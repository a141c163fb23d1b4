"""The bounded waits of the experts' products, run out on the GPU without a
fault: in the instrumented build every block's first copies are expected to
bring 16 bytes more than they do, so that the wait for them ends after a short
limit. The call returns, says so in the device error word, and the next one is
right."""

import pytest
import torch

import segmented_radix_top_gb300 as st
from tests.test_gpu_rows_experts import ids_of
from tests.test_gpu_rows_matmul import eight_bits, whole

pytestmark = pytest.mark.gpu
SHORT_WAIT, DEFAULT_WAIT = 1 << 20, 1 << 31
BF16, F32 = 1, 2


@pytest.fixture(scope="module")
def instr():
    L = st.load_instrumented()
    yield L
    st.set_test_hooks(DEFAULT_WAIT, 0)


def calls(kind):
    """(result's shape, a call of an entry point of library L that writes it, the same through the package)"""
    tokens, k, experts, width, out = (2000, 2, 3, 640, 520) if kind != "few rows in 8 bits" else (20, 2, 8, 640, 520)
    groups = st.group_by_expert(ids_of(tokens, k, experts, 1, 0.1).cuda(), experts)
    n = tokens * k
    stream = torch.cuda.current_stream().cuda_stream
    if "8 bits" in kind:
        rows, weights, rs, ws = eight_bits(tokens, k, experts, width, out, True)
        own = st.expert_matmul(rows, weights, groups, row_scales=rs, weight_scales=ws, out_dtype=torch.float32)
        return own, lambda L, to: L.segtopk_expert_matmul_f8(
            rows.data_ptr(), n, width, width, rs.data_ptr(), rs.stride(0), weights.data_ptr(), experts, out, out * width, width,
            ws.data_ptr(), groups.offsets.data_ptr(), F32, to.data_ptr(), stream)
    rows, weights = whole(n, width, seed=1, dtype=torch.bfloat16), whole(experts, out, width, seed=2, dtype=torch.bfloat16)
    grad = whole(n, out, seed=3, dtype=torch.bfloat16)
    if kind == "weights' gradient":
        own = st.expert_matmul_backward(grad, rows, weights, groups, dtype=torch.float32)[1]
        return own, lambda L, to: L.segtopk_expert_matmul_weights(
            BF16, grad.data_ptr(), out, out, rows.data_ptr(), width, width, n, experts, groups.offsets.data_ptr(), F32,
            to.data_ptr(), stream)
    if kind == "transposed":
        own = st.expert_matmul(grad, weights.transpose(1, 2), groups, out_dtype=torch.float32)
        return own, lambda L, to: L.segtopk_expert_matmul(
            BF16, grad.data_ptr(), n, out, out, weights.data_ptr(), experts, width, out * width, 1, width,
            groups.offsets.data_ptr(), F32, to.data_ptr(), stream)
    own = st.expert_matmul(rows, weights, groups, out_dtype=torch.float32)
    return own, lambda L, to: L.segtopk_expert_matmul(
        BF16, rows.data_ptr(), n, width, width, weights.data_ptr(), experts, out, out * width, width, 1,
        groups.offsets.data_ptr(), F32, to.data_ptr(), stream)


@pytest.mark.parametrize("kind", ["16 bits", "transposed", "weights' gradient", "8 bits", "few rows in 8 bits"])
def test_wait_that_runs_out_sets_the_error_bit_and_returns(instr, kind):
    want, call = calls(kind)
    got = torch.empty_like(want)
    st.set_test_hooks(DEFAULT_WAIT, 0)
    assert call(instr, got) == 0 and torch.equal(got, want)
    assert st.read_device_error(lib=instr) == 0
    st.set_test_hooks(SHORT_WAIT, 16)
    try:
        assert call(instr, got) == 0
        err = st.read_device_error(lib=instr)
    finally:
        st.set_test_hooks(DEFAULT_WAIT, 0)
    assert err & 1, "the wait did not report running out (error word %#x)" % err
    # the context is usable, and nothing of that call is left behind
    got.fill_(7)
    assert call(instr, got) == 0 and torch.equal(got, want)
    assert st.read_device_error(lib=instr) == 0

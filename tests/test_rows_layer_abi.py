"""Host-only checks of layer norm, 8-bit rows, routing by groups and the
experts' products: constants, refusals of the C entry points and of the
binding. No call here reaches a launch."""
import ctypes

import pytest
import torch

import segmented_radix_top_gb300 as st
from segmented_radix_top_gb300 import _rows as R
from tests.test_abi import _header_define

OK, INVALID, NOT_SUPPORTED, MISALIGNED = 0, 1, 3, 4
F16, BF16, F32, F64 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    st.build()
    return st.load()


def test_constants_match_the_header():
    assert R.MAX_GROUPS == _header_define("SEGTOPK_MAX_GROUPS")
    assert R.MAX_NORM_WIDTH == _header_define("SEGTOPK_MAX_NORM_WIDTH")


def test_route_groups_refusals(lib):
    def call(dtype=F32, logits=64, tokens=4, experts=8, stride=8, k=2, groups=4, kept=2, two=0, score=0, renormalize=1,
             bias=None, ids=128, weights=256):
        return lib.segtopk_route_groups(dtype, logits, tokens, experts, stride, k, groups, kept, two, score, renormalize, 1.0,
                                        bias, ids, weights, None)
    for bad in (dict(dtype=9), dict(score=2), dict(renormalize=2), dict(tokens=-1), dict(experts=0), dict(k=0), dict(stride=-8),
                dict(logits=None), dict(ids=None), dict(weights=None), dict(groups=0), dict(groups=3), dict(kept=0), dict(kept=5),
                dict(two=2), dict(two=-1), dict(k=5), dict(kept=1, k=3)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dtype=F64), dict(experts=2048, k=2), dict(experts=64, groups=64), dict(experts=128, k=33, kept=4),
                dict(tokens=2 ** 30, k=2)):
        assert call(**bad) == NOT_SUPPORTED, bad
    for bad in (dict(logits=66), dict(ids=130), dict(weights=254), dict(bias=66)):
        assert call(**bad) == MISALIGNED, bad
    assert call(tokens=0, logits=None, ids=None, weights=None) == OK
    assert lib.segtopk_last_launch_count() == 0


def test_layer_norm_refusals(lib):
    def forward(dtype=F32, x=64, rows=4, width=8, stride=8, weight_dtype=F32, weight=128, bias=None, eps=1e-5, out=512, mean=1024,
                rstd=2048):
        return lib.segtopk_layer_norm(dtype, x, rows, width, stride, weight_dtype, weight, bias, eps, out, mean, rstd, None)

    def backward(dtype=F32, grad=64, grad_stride=8, x=64, rows=4, width=8, stride=8, weight_dtype=F32, weight=128, mean=1024,
                 rstd=2048, out=512, grad_weight=4096, grad_bias=8192, space=16384, size=1 << 30):
        return lib.segtopk_layer_norm_backward(dtype, grad, grad_stride, x, rows, width, stride, weight_dtype, weight, mean, rstd,
                                               out, grad_weight, grad_bias, space, size, None)

    for call in (forward, backward):
        for bad in (dict(dtype=-1), dict(dtype=6), dict(weight_dtype=6), dict(rows=-1), dict(width=0), dict(stride=-1),
                    dict(x=None), dict(weight=None), dict(mean=None), dict(rstd=None), dict(out=None)):
            assert call(**bad) == INVALID, (call, bad)
        for bad in (dict(dtype=F64), dict(dtype=F32, weight_dtype=F16), dict(dtype=F16, weight_dtype=BF16), dict(rows=2 ** 31),
                    dict(width=16385)):
            assert call(**bad) == NOT_SUPPORTED, (call, bad)
        for bad in (dict(x=66), dict(weight=130), dict(mean=1026), dict(rstd=2050), dict(out=514), dict(dtype=F16, x=65)):
            assert call(**bad) == MISALIGNED, (call, bad)
    assert forward(eps=-1e-9) == forward(eps=float("nan")) == INVALID and forward(bias=66) == MISALIGNED
    assert forward(rows=0, x=None) == OK
    for bad in (dict(grad=None), dict(grad_stride=-1), dict(grad_weight=None), dict(grad_bias=None), dict(space=None), dict(size=255),
                dict(rows=0, grad_bias=None)):
        assert backward(**bad) == INVALID, bad
    for bad in (dict(grad=66), dict(grad_weight=4098), dict(grad_bias=8193), dict(space=16386)):
        assert backward(**bad) == MISALIGNED, bad
    assert lib.segtopk_last_launch_count() == 0
    need = lib.segtopk_layer_norm_backward_workspace_bytes
    assert need(0, 8) == need(-1, 8) == need(4, 0) == need(4, 16385) == need(2 ** 31, 8) == 0
    assert need(4, 8) == 4 * 2 * 8 * 4 and need(2 ** 31 - 1, 16384) > 0


def test_quantize_refusals(lib):
    def call(dtype=F32, x=64, rows=4, width=8, stride=8, values=129, scales=256):
        return lib.segtopk_quantize_rows(dtype, x, rows, width, stride, values, scales, None)
    for bad in (dict(dtype=-1), dict(dtype=6), dict(rows=-1), dict(width=0), dict(stride=-1), dict(x=None), dict(values=None),
                dict(scales=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dtype=F64), dict(rows=2 ** 31), dict(width=2 ** 20 + 1), dict(rows=2 ** 31 - 1, width=256)):
        assert call(**bad) == NOT_SUPPORTED, bad
    assert call(x=66) == call(scales=258) == call(dtype=F16, x=65) == MISALIGNED
    assert call(rows=0, x=None) == OK
    assert lib.segtopk_last_launch_count() == 0


def test_expert_matmul_refusals(lib):
    def f16(dtype=BF16, rows=64, n=4, width=8, stride=8, weights=128, experts=2, out_width=16, expert_stride=128, out_stride=8,
            in_stride=1, offsets=256, out_dtype=BF16, out=512):
        return lib.segtopk_expert_matmul(dtype, rows, n, width, stride, weights, experts, out_width, expert_stride, out_stride,
                                         in_stride, offsets, out_dtype, out, None)

    def f8(rows=64, n=4, width=16, stride=16, row_scales=4, scale_stride=1, weights=128, experts=2, out_width=16,
           expert_stride=256, out_stride=16, weight_scales=8, offsets=256, out_dtype=BF16, out=512):
        return lib.segtopk_expert_matmul_f8(rows, n, width, stride, row_scales, scale_stride, weights, experts, out_width,
                                            expert_stride, out_stride, weight_scales, offsets, out_dtype, out, None)

    for call in (f16, f8):
        for bad in (dict(rows=None), dict(n=-1), dict(width=0), dict(stride=-16), dict(stride=7), dict(weights=None),
                    dict(experts=0), dict(out_width=0), dict(expert_stride=96), dict(out_stride=7), dict(offsets=None),
                    dict(out_dtype=6), dict(out=None)):
            assert call(**bad) == INVALID, (call, bad)
        for bad in (dict(n=2 ** 31 - 256), dict(experts=1025),
                    dict(width=2 ** 20 + 16, stride=2 ** 21, out_stride=2 ** 21, expert_stride=2 ** 30),
                    dict(out_width=2 ** 20 + 1), dict(out_dtype=F64), dict(stride=2 ** 37)):
            assert call(**bad) == NOT_SUPPORTED, (call, bad)
        for bad in (dict(rows=72), dict(stride=20), dict(weights=136), dict(expert_stride=260), dict(out_stride=20),
                    dict(offsets=260), dict(out=513), dict(out_dtype=F32, out=514)):
            assert call(**{**bad, **({"expert_stride": 512} if "out_stride" in bad else {})}) == MISALIGNED, (call, bad)
        assert call(n=0, rows=None, out=None) == OK
    assert f16(dtype=9) == f16(in_stride=2) == f16(out_stride=1, in_stride=8) == INVALID
    for bad in (dict(dtype=F32), dict(width=12, stride=16, out_stride=16, expert_stride=256),
                dict(out_width=12, out_stride=1, in_stride=16)):
        assert f16(**bad) == NOT_SUPPORTED, bad
    assert f16(out_stride=1, in_stride=20, expert_stride=512) == MISALIGNED
    assert f8(width=24, stride=32, out_stride=32, expert_stride=512) == NOT_SUPPORTED
    assert f8(row_scales=None) == f8(weight_scales=None) == f8(scale_stride=-1) == INVALID
    assert f8(row_scales=6) == f8(weight_scales=6) == MISALIGNED
    assert lib.segtopk_last_launch_count() == 0


def test_expert_matmul_weights_refusals(lib):
    def call(dtype=BF16, a=64, a_width=8, a_stride=8, b=128, b_width=16, b_stride=16, n=4, experts=2, offsets=256,
             out_dtype=BF16, out=512):
        return lib.segtopk_expert_matmul_weights(dtype, a, a_width, a_stride, b, b_width, b_stride, n, experts, offsets, out_dtype,
                                                 out, None)
    for bad in (dict(dtype=9), dict(a=None), dict(b=None), dict(a_width=0), dict(b_width=0), dict(a_stride=7), dict(b_stride=8),
                dict(n=-1), dict(experts=0), dict(offsets=None), dict(out=None), dict(out_dtype=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dtype=F32), dict(out_dtype=F64), dict(a_width=12, a_stride=16), dict(b_width=12), dict(experts=1025),
                dict(n=2 ** 31), dict(a_width=2 ** 20 + 8, a_stride=2 ** 21)):
        assert call(**bad) == NOT_SUPPORTED, bad
    for bad in (dict(a=72), dict(b=136), dict(a_stride=12), dict(b_stride=20), dict(offsets=260), dict(out=513)):
        assert call(**bad) == MISALIGNED, bad
    assert lib.segtopk_last_launch_count() == 0


def test_the_binding_refuses_what_it_cannot_pass_on(lib):
    x, ids = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    w, v = torch.ones(16), torch.zeros(4)
    groups = st.ExpertGroups(torch.zeros(9, dtype=torch.int64), ids, torch.zeros(8, dtype=torch.int32))
    rows, weights = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(8, 32, 16, dtype=torch.bfloat16)
    r8, w8 = rows.to(torch.float8_e4m3fn), weights.to(torch.float8_e4m3fn)
    for call in (lambda: st.route(x, 2, num_groups=4),                # not on a GPU
                 lambda: st.route(x, 2, num_groups=4, group_score="mean"),
                 lambda: st.layer_norm(x, w),
                 lambda: st.layer_norm(x, w.double()),
                 lambda: st.layer_norm(x, w[:8]),
                 lambda: st.layer_norm(x.double(), w),
                 lambda: st.layer_norm(x[0], w),
                 lambda: st.layer_norm_backward(x, x, w, v, v),
                 lambda: st.layer_norm_backward(x[:3], x, w, v, v),
                 lambda: st.layer_norm_backward(x, x.half(), w, v, v),
                 lambda: st.quantize_rows(x),
                 lambda: st.quantize_rows(x.long()),
                 lambda: st.expert_matmul(rows, weights, groups),
                 lambda: st.expert_matmul(rows.float(), weights.float(), groups),
                 lambda: st.expert_matmul(rows, weights.half(), groups),
                 lambda: st.expert_matmul(rows, weights[:, :, :8], groups),
                 lambda: st.expert_matmul(rows, weights[0], groups),
                 lambda: st.expert_matmul(r8, w8, groups),            # scales are wanted
                 lambda: st.expert_matmul(r8, w8, groups, row_scales=torch.ones(8, 1)),
                 lambda: st.expert_matmul(rows, weights, groups, row_scales=torch.ones(8, 1), weight_scales=torch.ones(8, 1, 1)),
                 lambda: st.expert_matmul_backward(rows, rows, weights, groups),
                 lambda: st.expert_matmul_backward(r8, r8, w8, groups)):
        with pytest.raises(ValueError):
            call()


def test_entry_points_take_their_declared_arguments(lib):
    for name in ("route_groups", "layer_norm", "layer_norm_backward", "quantize_rows", "expert_matmul", "expert_matmul_f8",
                 "expert_matmul_weights"):
        fn = getattr(lib, "segtopk_" + name)
        assert fn.restype is ctypes.c_int and fn.argtypes[-1] is ctypes.c_void_p
    assert lib.segtopk_layer_norm_backward_workspace_bytes.restype is ctypes.c_size_t

"""Host-only checks of the row operators: constants, refusals of the C entry
points and of the binding. No call here reaches a launch."""
import ctypes

import pytest
import torch

import segmented_radix_top_gb300 as st
from segmented_radix_top_gb300 import _rows as R
from tests.test_abi import _header_define

OK, INVALID, NOT_SUPPORTED, MISALIGNED = 0, 1, 3, 4
F16, F32, F64 = 0, 2, 3


@pytest.fixture(scope="module")
def lib():
    st.build()
    return st.load()


def test_constants_match_the_header():
    assert R.MAX_EXPERTS == _header_define("SEGTOPK_MAX_EXPERTS")
    assert R.ROUTE_MAX_K == _header_define("SEGTOPK_ROUTE_MAX_K")
    assert R.DEVICE_ERROR_INDEX == _header_define("SEGTOPK_DEVICE_ERROR_INDEX")


def route(lib, dtype=F32, logits=64, tokens=4, experts=8, stride=8, k=2, score=0, renormalize=1, bias=None, ids=128,
          weights=256, backward=False):
    if backward:
        return lib.segtopk_route_backward(dtype, weights, logits, tokens, experts, stride, k, ids, score, renormalize,
                                          1.0, 512, None)
    return lib.segtopk_route(dtype, logits, tokens, experts, stride, k, score, renormalize, 1.0, bias, ids, weights,
                             None)


@pytest.mark.parametrize("backward", [False, True])
def test_route_refusals(lib, backward):
    def call(**kw):
        return route(lib, backward=backward, **kw)
    for bad in (dict(dtype=9), dict(dtype=-1), dict(score=2), dict(renormalize=2), dict(tokens=-1), dict(experts=0),
                dict(k=0), dict(k=9), dict(stride=-8), dict(logits=None), dict(ids=None), dict(weights=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dtype=F64), dict(dtype=5), dict(experts=1025, k=2), dict(experts=64, k=33),
                dict(tokens=2 ** 30, k=2)):
        assert call(**bad) == NOT_SUPPORTED, bad
    for bad in (dict(logits=66), dict(dtype=F16, logits=65), dict(ids=130), dict(weights=254)):
        assert call(**bad) == MISALIGNED, bad
    assert call(tokens=0, logits=None, ids=None, weights=None) == OK
    assert lib.segtopk_last_launch_count() == 0


def test_route_refuses_a_misaligned_bias(lib):
    assert route(lib, bias=66) == MISALIGNED


def test_group_refusals(lib):
    def call(ids=64, id_bytes=4, slots=100, experts=8, offsets=128, rows=256, order=512, space=None, size=0):
        return lib.segtopk_group(ids, id_bytes, slots, experts, offsets, rows, order, space, size, None)
    for bad in (dict(id_bytes=2), dict(slots=-1), dict(experts=0), dict(offsets=None), dict(ids=None),
                dict(rows=None), dict(order=None), dict(slots=10 ** 6)):
        assert call(**bad) == INVALID, bad
    need = lib.segtopk_group_workspace_bytes(10 ** 6, 8)
    assert need > 0
    assert call(slots=10 ** 6, space=1024, size=need - 1) == INVALID
    for bad in (dict(experts=1025), dict(slots=2 ** 31)):
        assert call(**bad) == NOT_SUPPORTED, bad
    for bad in (dict(ids=66), dict(ids=68, id_bytes=8), dict(offsets=132), dict(rows=258), dict(order=513)):
        assert call(**bad) == MISALIGNED, bad
    assert lib.segtopk_last_launch_count() == 0


def test_workspace_bytes_cover_the_range(lib):
    group, grad = lib.segtopk_group_workspace_bytes, lib.segtopk_embedding_backward_workspace_bytes
    assert group(0, 8) == group(-1, 8) == group(2 ** 31, 8) == group(100, 0) == group(100, 1025) == 0
    assert group(2 ** 31 - 1, 1024) >= 1025 * 4 * 2
    assert grad(-1, 10, 10) == grad(10, 0, 10) == grad(10, 10, -1) == grad(10, 2 ** 31 - 1, 8) == 0
    # four index arrays for the sorted tokens at least
    assert grad(10 ** 6, 10 ** 5, 64) >= 4 * 4 * 10 ** 6


def test_dispatch_and_combine_refusals(lib):
    def dispatch(x=64, size=2, tokens=4, k=2, width=8, stride=8, rows=128, kept=256, out=512):
        return lib.segtopk_dispatch(x, size, tokens, k, width, stride, rows, kept, out, None)

    def combine(dtype=F32, values=64, tokens=4, k=2, width=8, stride=8, rows=128, weights=None, out=512):
        return lib.segtopk_combine(dtype, values, tokens, k, width, stride, rows, weights, out, None)

    def backward(dtype=F32, grad=64, grad_stride=8, values=128, stride=8, tokens=4, k=2, width=8, rows=256, kept=512,
                 weights=1024, grad_values=2048, grad_weights=4096):
        return lib.segtopk_combine_backward(dtype, grad, grad_stride, values, stride, tokens, k, width, rows, kept,
                                            weights, grad_values, grad_weights, None)

    for call in (dispatch, combine, backward):
        for bad in (dict(tokens=-1), dict(k=0), dict(width=-1), dict(stride=-1), dict(rows=None)):
            assert call(**bad) == INVALID, (call, bad)
        assert call(tokens=2 ** 30, k=2) == NOT_SUPPORTED
        assert call(rows=130) == MISALIGNED
        assert call(tokens=0) == OK
    for bad in (dict(x=None), dict(out=None), dict(kept=None), dict(size=3)):
        assert dispatch(**bad) == INVALID, bad
    assert dispatch(x=65) == dispatch(kept=260) == dispatch(size=8, out=516) == MISALIGNED
    for bad in (dict(values=None), dict(out=None), dict(dtype=7)):
        assert combine(**bad) == INVALID, bad
    assert combine(dtype=F64) == backward(dtype=4) == NOT_SUPPORTED
    assert combine(values=66) == combine(weights=129) == backward(grad=66) == backward(kept=516) == MISALIGNED
    for bad in (dict(grad=None), dict(values=None), dict(kept=None), dict(weights=None), dict(grad_values=None),
                dict(grad_weights=None), dict(grad_stride=-1), dict(dtype=-1)):
        assert backward(**bad) == INVALID, bad
    assert lib.segtopk_last_launch_count() == 0


def test_embedding_refusals(lib):
    def forward(dtype=F32, table=64, vocab=10, width=8, stride=8, tokens=128, size=8, n=4, out_dtype=F32, out=512):
        return lib.segtopk_embedding(dtype, table, vocab, width, stride, tokens, size, n, 1.0, out_dtype, out, None)

    def backward(dtype=F32, grad=64, stride=8, tokens=128, size=8, n=4, vocab=10, width=8, table_dtype=F32, out=512,
                 accumulate=0, space=1024, space_bytes=1 << 40):
        return lib.segtopk_embedding_backward(dtype, grad, stride, tokens, size, n, vocab, width, -1, 1.0, table_dtype,
                                              out, accumulate, space, space_bytes, None)

    for call in (forward, backward):
        for bad in (dict(size=2), dict(n=-1), dict(vocab=0), dict(width=-1), dict(stride=-1), dict(dtype=9),
                    dict(tokens=None), dict(out=None)):
            assert call(**bad) == INVALID, (call, bad)
        for bad in (dict(dtype=F64), dict(n=2 ** 31), dict(vocab=2 ** 31 - 1), dict(width=2 ** 20 + 1)):
            assert call(**bad) == NOT_SUPPORTED, (call, bad)
        for bad in (dict(tokens=132), dict(out=514)):
            assert call(**bad) == MISALIGNED, (call, bad)
        assert call(width=0) == OK
    assert forward(n=0) == OK and forward(table=None) == INVALID and forward(table=66) == MISALIGNED
    assert forward(out_dtype=F64) == backward(table_dtype=F64) == NOT_SUPPORTED
    assert backward(n=0, accumulate=1) == OK
    assert backward(accumulate=2) == backward(grad=None) == backward(space=None) == backward(space_bytes=64) == INVALID
    assert backward(space=1024 + 128) == MISALIGNED
    assert lib.segtopk_last_launch_count() == 0


def test_the_binding_refuses_what_it_cannot_pass_on(lib):
    x, ids, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    groups = st.ExpertGroups(torch.zeros(9, dtype=torch.int64), ids, torch.zeros(8, dtype=torch.int32))
    for call in (lambda: st.route(x, 2),                             # not on a GPU
                 lambda: st.route(x.double(), 2),
                 lambda: st.route(x[0], 2),
                 lambda: st.route(x, 2, score="relu"),
                 lambda: st.route_backward(w, x, ids),
                 lambda: st.route_backward(w.double(), x, ids),
                 lambda: st.route_backward(w, x, ids.long()),
                 lambda: st.group_by_expert(ids, 8),
                 lambda: st.group_by_expert(w, 8),
                 lambda: st.group_by_expert(ids[0], 8),
                 lambda: st.dispatch(x, groups),
                 lambda: st.dispatch(x[:3], groups),
                 lambda: st.combine(x, groups, w),                   # 8 rows are wanted
                 lambda: st.combine(torch.zeros(8, 8), groups, None),
                 lambda: st.combine(torch.zeros(8, 8), groups, w.half()),
                 lambda: st.combine_backward(x[:, :4], torch.zeros(8, 8), groups, w),
                 lambda: st.dispatch_backward(torch.zeros(8, 8, dtype=torch.int32), groups),
                 lambda: st.embedding(x, ids),
                 lambda: st.embedding(x, w),
                 lambda: st.embedding_backward(x, ids, 10),
                 lambda: st.embedding_backward(x, ids[:, 0], 10, padding_idx=10),
                 lambda: st.embedding_backward(x, ids[:, 0], 10, accumulate=True)):
        with pytest.raises(ValueError):
            call()


def test_entry_points_take_their_declared_arguments(lib):
    # every argument's type is declared: ctypes would pass a Python int as a C int
    for name in ("route", "route_backward", "group", "dispatch", "combine", "combine_backward", "embedding",
                 "embedding_backward"):
        fn = getattr(lib, "segtopk_" + name)
        assert fn.restype is ctypes.c_int and fn.argtypes[-1] is ctypes.c_void_p

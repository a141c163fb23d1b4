"""Inputs and outputs whose conjugation or negation torch has put off: such a
view shares another tensor's memory and only carries a mark."""
import pytest
import torch

import segmented_radix_top_gb300 as st

pytestmark = pytest.mark.gpu


def groups_of(tokens, k, experts):
    g = torch.Generator().manual_seed(tokens)
    return st.group_by_expert(torch.randint(-1, experts, (tokens, k), generator=g).cuda(), experts)


def complex_rows(tokens, width, dtype):
    g = torch.Generator().manual_seed(1)
    parts = torch.randint(-50, 50, (tokens, width, 2), generator=g).float()
    return torch.view_as_complex(parts.half() if dtype == torch.complex32 else parts).cuda()


@pytest.mark.parametrize("dtype", [torch.complex64, torch.complex32])
@pytest.mark.parametrize("width", [1, 5, 48])
def test_dispatch_of_conjugated_rows(width, dtype):
    groups = groups_of(13, 3, 6)
    wide = complex_rows(13, width + 6, dtype)
    for x in (wide, wide[:, 2:2 + width], wide[:1].expand(13, width + 6)):
        got = st.dispatch(x.conj(), groups)
        assert not got.is_conj()
        want = st.dispatch(x.conj().resolve_conj(), groups)
        assert torch.equal(torch.view_as_real(got), torch.view_as_real(want))
        assert torch.equal(got.imag, -st.dispatch(x, groups).imag)
    assert torch.equal(st.dispatch(wide.conj().imag, groups), -st.dispatch(wide.imag.contiguous(), groups))


@pytest.mark.parametrize("width", [7, 64])
def test_negated_views_of_every_input(width):
    neg = torch._neg_view
    g = torch.Generator().manual_seed(2)
    l, x, y = (torch.randn(n, width, generator=g).cuda() for n in (11, 11, 22))
    w = torch.rand(11, 2, generator=g).cuda()
    bias = torch.rand(width, generator=g).cuda()
    ids, _ = st.route(l, 2)
    groups = st.group_by_expert(ids, width)
    tokens = torch.randint(0, 11, (30,), generator=g).cuda()
    grad = torch.randn(30, width, generator=g).cuda()
    for call, inputs in (
            (lambda l, b: st.route(l, 2, bias=b), (l, bias)),
            (lambda w, l, i: st.route_backward(w, l, i), (w, l, ids)),
            (lambda i: st.group_by_expert(i, width), (ids,)),
            (lambda x: st.dispatch(x, groups), (x,)),
            (lambda y: st.dispatch_backward(y, groups), (y,)),
            (lambda y, w: st.combine(y, groups, w), (y, w)),
            (lambda x, y, w: st.combine_backward(x, y, groups, w), (x, y, w)),
            (lambda x, t: st.embedding(x, t), (x, tokens)),
            (lambda d, t: st.embedding_backward(d, t, 11), (grad, tokens))):
        want = call(*inputs)
        got = call(*(neg(-t) for t in inputs))
        for a, b in zip(*(r if isinstance(r, tuple) else (r,) for r in (got, want))):
            assert not a.is_neg() and torch.equal(a, b)


def test_such_outputs_are_refused():
    groups = groups_of(9, 2, 4)
    x = torch.zeros(9, 8, device="cuda")
    z = torch.zeros(9, 8, dtype=torch.complex64, device="cuda")
    with pytest.raises(ValueError):
        st.dispatch(z, groups, out=torch.zeros(18, 8, dtype=torch.complex64, device="cuda").conj())
    for call in (lambda out: st.dispatch(x, groups, out=out[:18]),
                 lambda out: st.dispatch_backward(x.repeat(2, 1), groups, out=out[:9]),
                 lambda out: st.combine(x.repeat(2, 1), groups, torch.ones(9, 2, device="cuda"), out=out[:9]),
                 lambda out: st.embedding(x, torch.zeros(20, dtype=torch.int64, device="cuda"), out=out),
                 lambda out: st.embedding_backward(x, torch.zeros(9, dtype=torch.int64, device="cuda"), 20,
                                                   grad_table=out)):
        call(torch.zeros(20, 8, device="cuda"))
        with pytest.raises(ValueError):
            call(torch._neg_view(torch.zeros(20, 8, device="cuda")))
    rows = groups._replace(row_of_slot=torch._neg_view(groups.row_of_slot))
    with pytest.raises(ValueError):
        st.dispatch(x, rows)

"""Expert routing against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref

pytestmark = pytest.mark.gpu
HOW = [("softmax", True, 1.0), ("softmax", False, 2.5), ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)]
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def logits_of(tokens, experts, dtype, seed, masked=False):
    g = torch.Generator().manual_seed(seed)
    l = 2 * torch.randn(tokens, experts, generator=g)
    if masked:
        l[torch.rand(l.shape, generator=g) < 0.4] = -np.inf
        l[tokens // 2] = -np.inf
    return l.to(dtype)


def check(l, k, score, renormalize, scale, on_gpu=None):
    """Forward and backward of one input against the definition."""
    on_gpu = l.cuda() if on_gpu is None else on_gpu
    tokens, experts = l.shape
    how = dict(score=score, renormalize=renormalize, scale=scale)
    ids, w = st.route(on_gpu, k, **how)
    x = ref.f64(l)
    want = ref.choose(x, k)
    assert np.array_equal(ids.cpu().numpy(), want)
    rel = ref.exp_bound(x, experts)
    exact = ref.weights_of(x, want, score, renormalize, scale)
    ref.within(w, exact, rel * np.abs(exact) + 1e-37)
    g = torch.randn(tokens, k, generator=torch.Generator().manual_seed(7))
    got = st.route_backward(g.cuda(), on_gpu, ids, **how)
    assert got.dtype == l.dtype
    exact, size = ref.logits_gradient(x, want, ref.f64(g), score, renormalize, scale)
    ref.within(got, exact, (4 * rel + 2 * k * ref.U32) * size + ref.rounded(l.dtype, np.abs(exact)) + 1e-37)


@pytest.mark.parametrize("score,renormalize,scale", HOW)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 8, 2), (9, 32, 8), (17, 60, 6), (5, 64, 1), (33, 129, 8),
                                              (8, 256, 32), (3, 511, 7), (2, 1024, 32), (40, 7, 7)])
def test_route(tokens, experts, k, dtype, score, renormalize, scale):
    check(logits_of(tokens, experts, dtype, tokens + experts), k, score, renormalize, scale)


@pytest.mark.parametrize("score,renormalize,scale", HOW)
@pytest.mark.parametrize("tokens,experts,k", [(20, 16, 6), (11, 33, 8), (6, 200, 4)])
def test_masked_experts_and_tokens_without_any(tokens, experts, k, score, renormalize, scale):
    l = logits_of(tokens, experts, torch.float32, 3, masked=True)
    l[1, :-2] = -np.inf  # fewer than k left
    check(l, k, score, renormalize, scale)
    ids, w = st.route(l.cuda(), k, score=score, renormalize=renormalize, scale=scale)
    assert (ids[tokens // 2] == -1).all() and (w[tokens // 2] == 0).all()


def test_lowest_values_of_the_type_are_no_mask():
    for dtype in DTYPES:
        l = torch.full((3, 40), torch.finfo(dtype).min, dtype=dtype)
        l[1, 30] = 1.0
        ids, w = st.route(l.cuda(), 3)
        assert ids.tolist() == [[0, 1, 2], [30, 0, 1], [0, 1, 2]]
        ref.within(w[0], np.full(3, 1 / 3), 4 * ref.U32)
        assert w[1].tolist() == [1.0, 0.0, 0.0]


def test_ties_go_to_the_lower_expert_and_zeros_are_equal():
    l = torch.zeros(4, 96)
    l[1] = -0.0
    l[2, ::2] = -0.0
    l[3] = torch.arange(96).float().floor_divide(24)
    ids, _ = st.route(l.cuda(), 5)
    assert ids.tolist() == [[0, 1, 2, 3, 4]] * 3 + [[72, 73, 74, 75, 76]]


@pytest.mark.parametrize("score,renormalize,scale", HOW)
def test_nan_and_infinities(score, renormalize, scale):
    l = logits_of(4, 50, torch.float32, 5)
    l[0, 20], l[0, 10] = float("nan"), float("inf")
    l[1, 49] = -float("nan")
    l[2, 3] = float("inf")
    ids, w = st.route(l.cuda(), 2, score=score, renormalize=renormalize, scale=scale)
    assert ids[0].tolist() == [20, 10] and ids[1, 0] == 49 and ids[2, 0] == 3
    assert torch.isnan(w[:2, 0]).all()
    if score == "softmax":
        assert torch.isnan(w[2, 0])  # inf - inf
    elif not renormalize:
        assert w[2, 0] == scale
    fine = st.route(l[3:].cuda(), 2, score=score, renormalize=renormalize, scale=scale)
    assert torch.equal(w[3:], fine[1])  # other tokens are as they are alone


def test_scores_that_vanish_still_have_ratios():
    # sigmoid(-200) is 0 in 32 bits; the chosen ones' shares are not
    l = torch.tensor([[-200.0, -201.0, -205.0, -300.0], [-90.0, -90.0, -400.0, -500.0]])
    check(l, 2, "sigmoid", True, 1.0)
    check(l, 2, "softmax", True, 1.0)


def test_one_expert_far_above():
    l = torch.full((2, 64), -100.0)
    l[:, 5] = 80.0
    for how in HOW:
        check(l, 3, *how)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts", [24, 256])
def test_bias_chooses_and_does_not_weigh(experts, score, renormalize):
    # scores + bias are set apart by more than 32 bits can confuse
    g = torch.Generator().manual_seed(experts)
    l = torch.randn(12, experts, generator=g)
    bias = torch.randperm(experts, generator=g).float() * 3
    bias[4] = -np.inf  # takes an expert out
    l[3] = -np.inf
    l[5, 6] = -np.inf
    ids, w = st.route(l.cuda(), 4, score=score, renormalize=renormalize, bias=bias.cuda())
    x = ref.f64(l)
    with np.errstate(invalid="ignore"):
        keys = np.where(x == -np.inf, -np.inf, ref.scores(x, score) + ref.f64(bias))
    want = ref.choose(keys, 4)
    assert np.array_equal(ids.cpu().numpy(), want) and not (want == 4).any()
    exact = ref.weights_of(x, want, score, renormalize, 1.0)
    ref.within(w, exact, ref.exp_bound(x, experts) * exact + 1e-37)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts,left,extra", [(64, 8, 8), (64, 3, 6), (40, 0, 1), (100, 5, 2)])
def test_columns_of_a_wider_tensor(experts, left, extra, dtype):
    wide = logits_of(21, left + experts + extra, dtype, 1)
    part = wide[:, left:left + experts]
    check(part, 4, "softmax", False, 1.0, on_gpu=wide.cuda()[:, left:left + experts])


def test_transposed_and_expanded_logits():
    l = logits_of(32, 48, torch.float32, 2)
    check(l, 4, "softmax", True, 1.0, on_gpu=l.t().contiguous().cuda().t())
    one = l[:1].expand(7, 48)
    check(one, 4, "sigmoid", True, 1.0, on_gpu=l[:1].cuda().expand(7, 48))


def test_no_tokens():
    l = torch.zeros(0, 16, device="cuda")
    ids, w = st.route(l, 2)
    assert ids.shape == w.shape == (0, 2)
    assert st.route_backward(w, l, ids).shape == (0, 16)


@pytest.mark.parametrize("score,renormalize,scale", HOW)
def test_gradient_against_differences(score, renormalize, scale):
    # central differences of the 64-bit weights with the choice held fixed:
    # off by their step squared and by cancellation, both below 1e-8
    l = logits_of(5, 12, torch.float32, 9)
    g = torch.randn(5, 3, generator=torch.Generator().manual_seed(1))
    ids, _ = st.route(l.cuda(), 3, score=score, renormalize=renormalize, scale=scale)
    got = ref.f64(st.route_backward(g.cuda(), l.cuda(), ids, score=score, renormalize=renormalize, scale=scale))
    x, at, step = ref.f64(l), ids.cpu().numpy().astype(np.int64), 1e-5
    for e in range(12):
        up, down = x.copy(), x.copy()
        up[:, e] += step
        down[:, e] -= step
        diff = ref.weights_of(up, at, score, renormalize, scale) - ref.weights_of(down, at, score, renormalize, scale)
        want = (ref.f64(g) * diff).sum(1) / (2 * step)
        assert np.abs(got[:, e] - want).max() < 1e-8 + 4 * ref.exp_bound(x, 12) * scale * np.abs(ref.f64(g)).sum(1).max()


def test_backward_ignores_slots_without_an_expert():
    l = logits_of(3, 20, torch.float32, 4)
    ids, _ = st.route(l.cuda(), 4)
    g = torch.randn(3, 4).cuda()
    gone = ids.clone()
    gone[1, 2:] = -1
    g[1, 2:] = float("nan")  # of a masked place
    gone[2] = -1
    got = st.route_backward(g, l.cuda(), gone)
    assert torch.isfinite(got).all() and (got[2] == 0).all()
    want, size = ref.logits_gradient(ref.f64(l), gone.cpu().numpy().astype(np.int64),
                                     np.nan_to_num(ref.f64(g)), "softmax", True, 1.0)
    ref.within(got, want, 4 * ref.exp_bound(ref.f64(l), 20) * size + 1e-37)


def test_ids_past_the_last_expert_are_not_followed():
    l = logits_of(2, 8, torch.float32, 4).cuda()
    ids = torch.tensor([[0, 8], [1 << 30, -5]], dtype=torch.int32, device="cuda")
    got = st.route_backward(torch.ones(2, 2, device="cuda"), l, ids, score="sigmoid", renormalize=False)
    assert (got[0, 1:] == 0).all() and got[0, 0] > 0 and (got[1] == 0).all()


def test_refusals():
    l = torch.zeros(4, 8, device="cuda")
    for bad in (dict(k=0), dict(k=9), dict(k=-3)):
        with pytest.raises(st.SegTopKError):
            st.route(l, **bad)
    with pytest.raises(st.SegTopKError):
        st.route(torch.zeros(2, 1025, device="cuda"), 2)
    with pytest.raises(ValueError):
        st.route(l, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        st.route(l, 2, bias=torch.zeros(8))
    with pytest.raises(ValueError):
        st.route(l, 2, score="tanh")


def test_many_tokens():
    l = logits_of(70001, 16, torch.bfloat16, 8)
    ids, w = st.route(l.cuda(), 2)
    want = torch.sort(l.float(), dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(ids.cpu().long(), want)
    exact = torch.softmax(l.double().gather(1, want), 1).numpy()
    ref.within(w, exact, ref.exp_bound(ref.f64(l), 16) * exact)

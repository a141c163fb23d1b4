"""Routing limited to groups of experts against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
SHAPES = [  # tokens, experts, k, groups, kept
    (1, 2, 1, 2, 1), (5, 8, 2, 4, 2), (100, 60, 6, 4, 2), (300, 64, 8, 8, 4), (257, 160, 6, 8, 3), (64, 256, 8, 8, 4),
    (33, 96, 3, 3, 1), (50, 31, 5, 31, 7), (40, 32, 32, 32, 32), (70, 1024, 16, 32, 5), (20, 1022, 8, 2, 1), (90, 500, 17, 5, 2),
    (60, 48, 6, 16, 16), (10, 7, 3, 1, 1), (200, 128, 20, 16, 9)]


def logits_of(tokens, experts, seed, dtype=torch.float32, masked=0.0, coarse=False):
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn(tokens, experts, generator=g)
    if coarse:  # many equal ones
        x = torch.round(2 * x) / 2
    x[torch.rand(tokens, experts, generator=g) < masked] = -np.inf
    if masked:
        x[torch.rand(tokens, generator=g) < 0.1] = -np.inf
    return x.to(dtype)


def group_scores(keys, groups, two):
    """NaN above all; an expert at -inf adds nothing."""
    parts = np.sort(np.where(np.isnan(keys), np.inf, keys).reshape(len(keys), groups, -1), axis=2)
    if not two or parts.shape[2] == 1:
        return parts[:, :, -1]
    second = np.where(parts[:, :, -2] == -np.inf, 0, parts[:, :, -2])
    return np.where(parts[:, :, -1] == -np.inf, -np.inf, parts[:, :, -1] + second)


def choose(keys, k, groups, kept, two):
    best = ref.choose(np.where(group_scores(keys, groups, two) == -np.inf, -1e300, group_scores(keys, groups, two)), kept)
    on = np.zeros((len(keys), groups), dtype=bool)
    np.put_along_axis(on, best, True, 1)
    return ref.choose(np.where(np.repeat(on, keys.shape[1] // groups, 1), keys, -np.inf), k)


def check_weights(got, l, ids, score, renormalize, scale):
    want = ref.weights_of(l, ids, score, renormalize, scale)
    ref.within(got, want, ref.exp_bound(l, l.shape[1]) * np.abs(want) + 2.0 ** -149)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,experts,k,groups,kept", SHAPES)
def test_best_groups(tokens, experts, k, groups, kept, dtype, score, renormalize):
    # logits are compared: equal ones tie to the lower group and expert
    for coarse, masked in ((False, 0.0), (True, 0.0), (True, 0.4)):
        x = logits_of(tokens, experts, experts + k, dtype, masked, coarse)
        ids, weights = st.route(x.cuda(), k, score=score, renormalize=renormalize, scale=2.5, num_groups=groups, groups_kept=kept)
        l = ref.f64(x)
        want = choose(l, k, groups, kept, False)
        assert np.array_equal(ids.cpu().numpy(), want)
        check_weights(weights, l, want, score, renormalize, 2.5)



@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["best", "best_two"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("tokens,experts,k,groups,kept", SHAPES)
def test_scores_and_biases(tokens, experts, k, groups, kept, biased, group_score, score):
    x = logits_of(tokens, experts, 3 * experts + k)
    bias = torch.randn(experts, generator=torch.Generator().manual_seed(5)) * (0.3 if score == "sigmoid" else 0.01)
    if biased and experts > 8:
        bias[1], bias[experts - 2] = -np.inf, -np.inf
    ids, weights = st.route(x.cuda(), k, score=score, bias=bias.cuda() if biased else None, num_groups=groups, groups_kept=kept,
                            group_score=group_score)
    l, two = ref.f64(x), group_score == "best_two"
    keys = ref.scores(l, score) + ref.f64(bias) if biased else ref.scores(l, score)
    want = choose(keys, k, groups, kept, two)
    # scores of 32 bits are a few roundings from these: rows in which the choice hangs on less are left out
    scores = group_scores(keys, groups, two)
    order = np.sort(scores, axis=1)[:, ::-1]
    near = np.zeros(len(l), dtype=bool)
    if kept < groups:
        near |= order[:, kept - 1] - order[:, kept] < 1e-6
    for t in range(len(l)):
        inside = np.sort(keys[t][np.repeat(scores[t] >= order[t, kept - 1], experts // groups)])[::-1]
        inside = inside[inside > -np.inf][:k + 1]
        near[t] |= bool((inside[:-1] - inside[1:] < 1e-6).any())
    got = ids.cpu().numpy()
    # spacings of a few hundred scores in a range of about one (softmax: of 1/100 and less)
    assert (score == "softmax" or near.mean() < 0.2) and np.array_equal(got[~near], want[~near])
    check_weights(weights, l, got, score, True, 1.0)


def test_tokens_with_few_experts_left():
    x = torch.full((4, 32), -np.inf)
    x[1, 20] = 1.0
    x[2, [3, 9, 30]] = torch.tensor([1.0, 2.0, 3.0])
    x[3, 0], x[3, 31] = float("nan"), 5.0
    ids, weights = st.route(x.cuda(), 4, num_groups=4, groups_kept=2)
    assert ids.tolist() == [[-1] * 4, [20, -1, -1, -1], [30, 9, -1, -1], [0, 31, -1, -1]]
    assert not weights[0].any() and weights[1].tolist() == [1, 0, 0, 0] and torch.isnan(weights[3, :2]).all()
    # best two: a lone expert's group has its score alone
    two, _ = st.route(x[:3].cuda(), 4, score="sigmoid", num_groups=4, groups_kept=2, group_score="best_two")
    assert two.tolist() == [[-1] * 4, [20, -1, -1, -1], [30, 9, -1, -1]]
    # 0.9 and 0.2 (sum 1.1) against 0.6 twice (1.2): by the best one group 0, by the sum group 1
    p = torch.tensor([[0.9, 0.2, 0.6, 0.6]], dtype=torch.float64)
    l = torch.log(p / (1 - p)).float().cuda()
    assert st.route(l, 1, score="sigmoid", num_groups=2, groups_kept=1)[0].tolist() == [[0]]
    assert st.route(l, 1, score="sigmoid", num_groups=2, groups_kept=1, group_score="best_two")[0].tolist() == [[2]]


def test_all_groups_kept_is_plain_routing():
    x = logits_of(3000, 160, 7, masked=0.3, coarse=True).cuda()
    for how in (dict(), dict(score="sigmoid", renormalize=False, scale=2.0)):
        plain = st.route(x, 6, **how)
        for kw in (dict(num_groups=8), dict(num_groups=8, groups_kept=8), dict(num_groups=1, groups_kept=1)):
            assert all(torch.equal(a, b) for a, b in zip(plain, st.route(x, 6, **how, **kw)))


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient(score, renormalize):
    # the chosen experts are held fixed; the softmax is over all experts, in groups or not
    x = logits_of(200, 96, 11)
    ids, weights = st.route(x.cuda(), 5, score=score, renormalize=renormalize, scale=1.5, num_groups=6, groups_kept=2)
    g = torch.randn(200, 5, generator=torch.Generator().manual_seed(1))
    got = st.route_backward(g.cuda(), x.cuda(), ids, score=score, renormalize=renormalize, scale=1.5)
    l, chosen, gd = ref.f64(x), ids.cpu().numpy().astype(np.int64), ref.f64(g)
    want, size = ref.logits_gradient(l, chosen, gd, score, renormalize, 1.5)
    ref.within(got, want, 4 * ref.exp_bound(l, 96) * size + 2.0 ** -149)
    # along a direction, by differences of the weights in 64 bits
    d, step = np.random.default_rng(3).standard_normal(l.shape), 1e-5
    ahead = [(gd * ref.weights_of(l + s * step * d, chosen, score, renormalize, 1.5)).sum() for s in (1, -1)]
    slope = (ahead[0] - ahead[1]) / (2 * step)
    off = (4 * ref.exp_bound(l, 96) * size * np.abs(d)).sum()
    assert abs((ref.f64(got) * d).sum() - slope) <= off + 1e-6 * (size * np.abs(d)).sum()


def test_strides_graphs_and_streams():
    wide = logits_of(700, 300, 1).cuda()
    for part in (wide[:, 8:168], wide[:, 3:163], wide[:1, :160].expand(700, 160)):
        want = st.route(part.contiguous(), 6, num_groups=8, groups_kept=3)
        assert all(torch.equal(a, b) for a, b in zip(want, st.route(part, 6, num_groups=8, groups_kept=3)))
    x = logits_of(700, 160, 2).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = st.route(x, 6, num_groups=8, groups_kept=3, group_score="best_two")
    x.copy_(logits_of(700, 160, 3))
    graph.replay()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = st.route(x, 6, num_groups=8, groups_kept=3, group_score="best_two", stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert st.route(x[:0], 6, num_groups=8, groups_kept=3)[0].shape == (0, 6)

"""Routing with a selection bias of the scores' own size: the choice is by
score + bias, and it is checked against keys in 64 bits. Two experts may
stand the other way round only where their keys differ by less than 32 bits
can hold apart."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = ref.U32


def keys_and_bound(l, bias, score):
    """Keys in 64 bits, and how far one held in 32 bits may be off: the
    exponential of a difference d rounded once by |d| + 4 units of its value
    (CUDA's bound for expf is two places), the sum by its terms' own errors
    (their mean |d| is at most the entropy, ln E) and by its longest chain of
    additions (E / 32 in a lane, five over the warp), then a reciprocal, a
    product and the addition of the bias."""
    with np.errstate(invalid="ignore"):
        s = np.where(l == -np.inf, 0, ref.scores(l, score))
    key = np.where(l == -np.inf, -np.inf, s + bias)
    experts = l.shape[1]
    if score == "softmax":
        with np.errstate(invalid="ignore"):
            d = np.where(np.isfinite(l), np.abs(l - l.max(1, keepdims=True)), 0)
        units = d + 4 + np.log(experts) + 4 + experts / 32 + 5 + 3
    else:  # an exponential, an addition, a division
        units = 4 + 3
    off = 1.01 * U * (units * s + np.abs(np.where(np.isfinite(key), key, 0))) + 2.0 ** -147
    return key, off


def wrong(ids, l, bias, score):
    """Whether a choice `ids` breaks the definition anywhere."""
    key, off = keys_and_bound(l, bias, score)
    for t in range(len(l)):
        ranked = sorted((e for e in range(l.shape[1]) if key[t, e] > -np.inf), key=lambda e: (-key[t, e], e))
        chosen = [e for e in ids[t] if e >= 0]
        if len(chosen) != min(len(ranked), len(ids[t])) or list(ids[t][:len(chosen)]) != chosen:
            return True
        if len(set(chosen)) != len(chosen) or any(key[t, e] == -np.inf for e in chosen):
            return True
        rest = [e for e in ranked if e not in chosen]
        for i, e in enumerate(chosen):
            behind = np.array(chosen[i + 1:] + rest, dtype=int)
            if (key[t, e] + off[t, e] < key[t, behind] - off[t, behind]).any():
                return True
            same = behind[(l[t, behind] == l[t, e]) & (bias[behind] == bias[e])]
            if (same < e).any():
                return True
    return False


def inputs(tokens, experts, kind, dtype):
    g = torch.Generator().manual_seed(experts + tokens)
    l = (1.5 * torch.randn(tokens, experts, generator=g)).to(dtype)
    if kind == "small":  # of the size that trained routers have
        bias = 0.1 * torch.rand(experts, generator=g) - 0.05
    elif kind == "zeros":
        bias = torch.zeros(experts)
    elif kind == "ties":  # equal logits and equal biases, more of them than the list of candidates holds
        l = (torch.randint(0, 2, (tokens, experts), generator=g) * 2.0).to(dtype)
        bias = torch.randint(0, 2, (experts,), generator=g) / 64.0
    else:  # masked in either way
        bias = 0.1 * torch.rand(experts, generator=g) - 0.05
        bias[torch.rand(experts, generator=g) < 0.2] = -np.inf
        l[torch.rand(l.shape, generator=g) < 0.3] = -np.inf
        l[1] = -np.inf
    return l, bias


KINDS = ["small", "zeros", "ties", "masked"]
# k on both sides of the limits of the list of candidates (k * share > 12 and k <= 16)
SIZES = [(9, 8, 2), (21, 64, 6), (21, 64, 7), (17, 100, 8), (33, 256, 1), (33, 256, 2), (33, 256, 8), (9, 256, 16),
         (9, 256, 17), (5, 1024, 32), (5, 1000, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,experts,k", SIZES)
def test_choice(tokens, experts, k, kind, dtype, score):
    l, bias = inputs(tokens, experts, kind, dtype)
    x, b = ref.f64(l), ref.f64(bias)
    ids, w = st.route(l.cuda(), k, score=score, renormalize=False, bias=bias.cuda())
    got = ids.cpu().numpy()
    assert not wrong(got, x, b, score)
    exact = ref.weights_of(x, got, score, False, 1.0)
    ref.within(w, exact, ref.exp_bound(x, experts) * exact + 1e-37)
    wide = torch.zeros(tokens, experts + 3, dtype=dtype, device="cuda")
    wide[:, 1:1 + experts] = l.cuda()
    again = st.route(wide[:, 1:1 + experts], k, score=score, renormalize=False, bias=bias.cuda())
    assert torch.equal(again[0], ids) and torch.equal(again[1], w)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,k", [s for s in SIZES if s[2] > 1])
def test_the_check_sees_a_wrong_key(tokens, experts, k, score):
    l, bias = inputs(tokens, experts, "small", torch.float32)
    x, b = ref.f64(l), ref.f64(bias)
    s = ref.scores(x, score)
    assert not wrong(ref.choose(s + b, k), x, b, score)
    assert wrong(ref.choose(np.broadcast_to(b, x.shape), k), x, b, score)  # the score left out
    assert wrong(ref.choose(x + b, k), x, b, score) or score == "softmax" and experts < 64  # the logit in its place
    if experts >= 64:  # the bias left out, or a sum left out
        assert wrong(ref.choose(s, k), x, b, score)
    l, bias = inputs(tokens, experts, "ties", torch.float32)
    x, b = ref.f64(l), ref.f64(bias)
    up = ref.choose((ref.scores(x, score) + b)[:, ::-1], k)
    assert wrong(experts - 1 - up, x, b, score)  # ties to the higher expert


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_below_the_normal_numbers_are_compared(score, dtype):
    # e^-90 and e^-88.5 are no normal numbers of 32 bits, and different
    l = torch.tensor([[0.0, -90.0, -88.5], [-89.5, 0.0, -89.0], [-100.0, -101.0, -99.0]], dtype=dtype).cuda()
    ids, _ = st.route(l, 2, score=score, bias=torch.zeros(3, device="cuda"))
    assert ids.tolist() == [[0, 2], [1, 2], [2, 0]]


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 3, 6])
@pytest.mark.parametrize("experts", [8, 200])
def test_a_bias_of_minus_infinity_wins_over_nan(experts, k):
    bias = torch.zeros(experts)
    bias[1] = bias[7] = -np.inf
    l = 0.01 * torch.arange(experts).float().expand(4, experts).clone()
    l[0, 5] = float("nan")
    l[1, 7] = float("nan")
    l[2, 4] = float("inf")
    l[3, 1] = float("inf")
    left = [e for e in range(experts) if e not in (1, 7)]
    ids, _ = st.route(l.cuda(), k, score="softmax", bias=bias.cuda())
    assert ids.tolist() == [left[:k]] * 4  # every score of such a row is NaN
    ids, _ = st.route(l.cuda(), k, score="sigmoid", bias=bias.cuda())
    down = left[::-1]
    assert ids.tolist() == [([5] + [e for e in down if e != 5])[:k], down[:k],
                            ([4] + [e for e in down if e != 4])[:k], down[:k]]

"""Accuracy of the scores that routing weighs by, where they are far below the
largest one."""
import numpy as np
import pytest
import torch

import segmented_radix_top_gb300 as st
from tests import rows_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,k", [(6, 30, 1), (9, 128, 4), (5, 256, 8), (3, 1024, 32)])
def test_gradient_of_experts_far_below_the_best(tokens, experts, k):
    # Whole numbers, so that differences of logits are exact, down to where
    # the softmax is no normal number of 32 bits (e^-102). A gradient is
    # -s_e times a sum of the k products; in units of 2^-24 the exponential
    # is off by 4 (two places), the softmax's sum by 4 of its terms and its
    # additions (experts / 32 in a lane, five over the warp) and it divides
    # twice, the k products by an exponential, a division, a scale and a
    # product, and by their sum's 5 additions; two more products at the end.
    g = torch.Generator().manual_seed(experts)
    l = -torch.randint(1, 103, (tokens, experts), generator=g).float()
    l[torch.arange(tokens), torch.randint(0, experts, (tokens,), generator=g)] = 0.0
    ids, w = st.route(l.cuda(), k, renormalize=False)
    gw = torch.rand(tokens, k, generator=g) + 0.5
    got = st.route_backward(gw.cuda(), l.cuda(), ids, renormalize=False)
    x = ref.f64(l)
    want, size = ref.logits_gradient(x, ids.cpu().numpy().astype(np.int64), ref.f64(gw), "softmax", False, 1.0)
    units = 4 + 2 * (4 + experts / 32 + 5 + 1) + 4 + 3 + 5 + 2
    ref.within(got, want, 1.01 * units * ref.U32 * size + 2.0 ** -146)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("spread", [0.0, 1.0, 4.0])
@pytest.mark.parametrize("tokens,experts,k", [(40, 16, 2), (40, 256, 8), (10, 1024, 32)])
def test_weights_of_the_whole_softmax(tokens, experts, k, spread, dtype):
    # in units of 2^-24: the chosen term's exponential, 4, and its rounded
    # difference, |d|; the sum's terms, 4 and their mean |d|, which is at
    # most ln(experts), each twice over (the difference and its product with
    # log2 e); the additions; a division and a scale
    l = (spread * torch.randn(tokens, experts, generator=torch.Generator().manual_seed(1))).to(dtype)
    ids, w = st.route(l.cuda(), k, renormalize=False, scale=1.5)
    x, at = ref.f64(l), ids.cpu().numpy().astype(np.int64)
    exact = ref.weights_of(x, at, "softmax", False, 1.5)
    d = x.max(1, keepdims=True) - np.take_along_axis(x, at, 1)
    units = 4 + d + 4 + 2.25 * np.log(experts) + experts / 32 + 5 + 2
    ref.within(w, exact, 1.01 * units * ref.U32 * exact)


@pytest.mark.parametrize("k", [1, 3, 8])
def test_sigmoids_near_their_ends(k):
    # s (1 - s) is no normal number of 32 bits beyond 87 on either side. In
    # units of 2^-24: an exponential 4, an addition, a division for each of the
    # two factors, and a scale and two products.
    experts = 40
    l = (torch.arange(6 * experts).reshape(6, experts) * 37 % 206 - 103).float()
    ids, w = st.route(l.cuda(), k, score="sigmoid", renormalize=False)
    ids[:, 0] = l.argmin(1).cuda()  # one at the lower end, k - 1 at the upper one
    gw = torch.rand(6, k, generator=torch.Generator().manual_seed(k)) + 0.5
    got = st.route_backward(gw.cuda(), l.cuda(), ids, score="sigmoid", renormalize=False)
    x, at = ref.f64(l), ids.cpu().numpy().astype(np.int64)
    want, size = ref.logits_gradient(x, at, ref.f64(gw), "sigmoid", False, 1.0)
    ref.within(got, want, 1.01 * 15 * ref.U32 * size + 2.0 ** -146)
    low = l - 90  # all of them
    ids, w = st.route(low.clamp(max=-50).cuda(), k, score="sigmoid", renormalize=False, scale=2.0)
    x, at = ref.f64(low.clamp(max=-50)), ids.cpu().numpy().astype(np.int64)
    exact = ref.weights_of(x, at, "sigmoid", False, 2.0)
    ref.within(w, exact, 1.01 * 7 * ref.U32 * exact + 2.0 ** -146)

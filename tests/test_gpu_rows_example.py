"""The operators together, as examples/sparse_layer.py uses them: the model's
gradients against torch's own in 64 bits, and training on a text with a rule."""
import pytest
import torch

from examples import sparse_layer

pytestmark = pytest.mark.gpu


def plain(model, tokens):
    """The same model by torch operations that autograd differentiates, in 64 bits, with the same choice of experts."""
    p = {n: v.detach().double().requires_grad_() for n, v in model.named_parameters()}
    x = p["table"][tokens] * p["table"].shape[1] ** 0.5
    logits = x @ p["router"]
    best, ids = logits.topk(model.k, 1)
    weights = torch.softmax(best, 1)
    every = torch.einsum("teh,ehw->tew", torch.nn.functional.gelu(torch.einsum("tw,ewh->teh", x, p["up"])), p["down"])
    chosen = every.gather(1, ids[..., None].expand(-1, -1, x.shape[1]))
    return (x + (weights[..., None] * chosen).sum(1)) @ p["head"], p, ids


def test_gradients_of_the_whole_model():
    model = sparse_layer.SparseModel(vocab=60, width=32, hidden=48, experts=6, k=2, seed=3)
    g = torch.Generator(device="cuda").manual_seed(2)
    tokens, following = sparse_layer.text(200, 60, g)
    torch.nn.functional.cross_entropy(model(tokens), following).backward()
    logits, p, _ = plain(model, tokens)
    torch.nn.functional.cross_entropy(logits, following).backward()
    # torch's products round to 32 bits over sums of at most 200 terms each,
    # five products deep
    for name, value in model.named_parameters():
        off = (value.grad.double() - p[name].grad).norm() / p[name].grad.norm()
        assert off < 5 * 200 * 2.0 ** -24, name


def test_it_learns_and_samples():
    losses, right = sparse_layer.train(steps=60)
    # 0.9 of the tokens by the rule, the others uniform: the entropy is 0.9 ln(1 / 0.9) + 0.1 ln(512 / 0.1) = 0.95
    assert losses[0] > 5 and losses[-1] < 2.5
    assert right > 0.7

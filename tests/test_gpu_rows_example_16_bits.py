"""The example's model in 16 bits, whose experts' products are the package's:
its gradients against torch's in 64 bits, and that it runs."""
import pytest
import torch

from examples import sparse_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradients_of_the_whole_model(dtype):
    model = sparse_layer.SparseModel(vocab=60, width=32, hidden=48, experts=6, k=2, seed=3, dtype=dtype)
    tokens, _ = sparse_layer.text(200, 60, torch.Generator(device="cuda").manual_seed(2))
    grad = torch.randn(200, 60, generator=torch.Generator().manual_seed(4)).to(dtype).cuda()
    out = model(tokens)
    out.backward(grad)
    p = {n: v.detach().double().requires_grad_() for n, v in model.named_parameters()}
    x = p["table"][tokens] * p["table"].shape[1] ** 0.5
    # the choice that the model made
    rounded = sparse_layer.st.embedding(model.table.detach(), tokens, scale=model.table.shape[1] ** 0.5)
    ids = sparse_layer.st.route(rounded @ model.router.detach(), model.k)[0].long()
    weights = torch.softmax((x @ p["router"]).gather(1, ids), 1)
    hidden = torch.nn.functional.gelu(torch.einsum("tw,tkwh->tkh", x, p["up"][ids]))
    y = x + torch.einsum("tkh,tkhw,tk->tw", hidden, p["down"][ids], weights)
    want = y @ p["head"]
    want.backward(grad.double())
    # eight results in 16 bits on the way to the logits and as many back, each off by half a unit of its value;
    # relative to norms each adds its own, the sum x + ... takes out none, and gelu's slope is at most 1.13: a factor of
    # 2 for it and the weights' differences
    bound = 16 * 2 * torch.finfo(dtype).eps / 2
    assert float((out.detach().double() - want.detach()).norm() / want.detach().norm()) <= bound
    for name, value in model.named_parameters():
        assert float((value.grad.double() - p[name].grad).norm() / p[name].grad.norm()) <= bound, name


def test_it_runs_and_samples():
    losses, right = sparse_layer.train(steps=3, dtype=torch.bfloat16)
    assert len(losses) == 3 and all(torch.isfinite(torch.tensor(losses))) and 0 <= right <= 1

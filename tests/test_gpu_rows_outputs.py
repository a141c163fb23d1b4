"""Given outputs and torch's autograd: a write counts as a change of the
tensor, and a tensor that autograd differentiates is no output."""
import pytest
import torch

import segmented_radix_top_gb300 as st

pytestmark = pytest.mark.gpu


def calls():
    """Name, shape of the output, and the call that writes it."""
    ids = torch.tensor([[0, 2], [1, -1], [2, 0]], dtype=torch.int32, device="cuda")
    groups = st.group_by_expert(ids, 3)
    x, y = torch.ones(3, 8, device="cuda"), torch.ones(6, 8, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    tokens = torch.tensor([4, 0, 4], device="cuda")
    return [("dispatch", (6, 8), lambda out: st.dispatch(x, groups, out=out)),
            ("dispatch_backward", (3, 8), lambda out: st.dispatch_backward(y, groups, out=out)),
            ("combine", (3, 8), lambda out: st.combine(y, groups, w, out=out)),
            ("embedding", (3, 8), lambda out: st.embedding(y, tokens, out=out)),
            ("embedding_backward", (5, 8), lambda out: st.embedding_backward(x, tokens, 5, grad_table=out)),
            ("accumulate", (5, 8), lambda out: st.embedding_backward(x, tokens, 5, grad_table=out, accumulate=True))]


NAMES = ["dispatch", "dispatch_backward", "combine", "embedding", "embedding_backward", "accumulate"]


@pytest.mark.parametrize("name", NAMES)
def test_autograd_sees_that_a_saved_tensor_was_written(name):
    _, shape, call = [c for c in calls() if c[0] == name][0]
    saved = torch.ones(shape, device="cuda")
    w = torch.ones(shape, device="cuda", requires_grad=True)
    loss = (w * saved).sum()
    before = saved._version
    assert call(saved.detach()) is not None  # a view shares its base's count of changes
    assert saved._version == before + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_that_autograd_differentiates_is_refused(name):
    _, shape, call = [c for c in calls() if c[0] == name][0]
    leaf = torch.ones(shape, device="cuda", requires_grad=True)
    for out in (leaf, leaf * 2):
        with pytest.raises(ValueError):
            call(out)
        assert (out.detach() == out.detach().flatten()[0]).all()  # nothing was written
    with torch.no_grad():
        before = leaf._version
        assert call(leaf) is leaf and leaf._version == before + 1


def test_a_refused_call_changes_nothing():
    _, shape, call = calls()[0]
    for bad in (torch.zeros(7, 8, device="cuda"), torch.zeros(shape, device="cuda").half()):
        with pytest.raises(ValueError):
            call(bad)
        assert bad._version == 0


def test_outputs_of_inference_mode():
    with torch.inference_mode():
        for name, shape, call in calls():
            out = torch.zeros(shape, device="cuda")
            assert call(out) is out, name

"""The decoding calls and autograd: no gradient or tangent is dropped in silence, and what is written in place counts as
a new version of its tensor."""
import pytest
import torch
from torch.autograd import forward_ad

import gated_delta_rule_50_gb300 as gdn
from test_decode_refusals import step_args

pytestmark = pytest.mark.gpu


def beam_args():
    return torch.randn(2, 3, 50, device="cuda"), torch.zeros(2, 3, device="cuda")


PARENTS = dict(dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "state"])
def test_tangents_are_refused(name):
    a = step_args("cuda")
    before = a["state"].clone()
    with forward_ad.dual_level():
        a[name] = forward_ad.make_dual(a[name], torch.ones_like(a[name]))
        with pytest.raises(ValueError, match="tangent|gradient|backward"):
            gdn.recurrent_gated_delta_rule(**a)
        with torch.no_grad(), pytest.raises(ValueError):
            gdn.tree_gated_delta_rule(*[a[n] for n in ("q", "k", "v", "g", "beta")], torch.full((2, 1), -1, **PARENTS), a["state"])
    assert torch.equal(forward_ad.unpack_dual(a["state"]).primal if name == "state" else a["state"], before)


def test_beam_and_reorder_tangents_are_refused():
    x, s = beam_args()
    parents = torch.zeros(2, 3, **PARENTS)
    with forward_ad.dual_level():
        with pytest.raises(ValueError):
            gdn.beam_search_step(forward_ad.make_dual(x, torch.ones_like(x)), s)
        with pytest.raises(ValueError):
            gdn.beam_search_step(x, forward_ad.make_dual(s, torch.ones_like(s)))
        with pytest.raises(ValueError):
            gdn.reorder_states(forward_ad.make_dual(torch.zeros(6, 4, device="cuda"), torch.ones(6, 4, device="cuda")), parents)


def test_beam_and_reorder_gradients_are_refused():
    x, s = beam_args()
    for kw in (dict(logits=x.clone().requires_grad_(), scores=s), dict(logits=x, scores=s.clone().requires_grad_())):
        with pytest.raises(ValueError, match="backward"):
            gdn.beam_search_step(**kw)
        with torch.no_grad():
            got = gdn.beam_search_step(**kw)
        assert all(torch.equal(a, b) for a, b in zip(got, gdn.beam_search_step(x, s)))
    leaf = torch.randn(6, 4, device="cuda").requires_grad_()
    before = leaf.detach().clone()
    for states in (leaf, [torch.zeros(6, 4, device="cuda"), leaf]):
        with pytest.raises(ValueError, match="backward"):
            gdn.reorder_states(states, torch.zeros(2, 3, **PARENTS))
    assert torch.equal(leaf, before)


def test_out_state_gradient_is_refused():
    a = step_args("cuda")
    out = torch.zeros(2, 4, 64, 64, device="cuda").requires_grad_()
    with pytest.raises(ValueError, match="backward"):
        gdn.recurrent_gated_delta_rule(**a, out_state=out)


def test_versions():
    a = step_args("cuda")
    state = a["state"]
    v0 = state._version
    gdn.recurrent_gated_delta_rule(**a)
    assert state._version == v0 + 1
    out = torch.zeros(2, 4, 64, 64, device="cuda")
    gdn.recurrent_gated_delta_rule(**a, out_state=out)
    assert state._version == v0 + 1 and out._version == 1  # only read; written
    gdn.tree_gated_delta_rule(*[a[n] for n in ("q", "k", "v", "g", "beta")], torch.full((2, 1), -1, **PARENTS), state)
    assert state._version == v0 + 1
    pool = torch.zeros(6, 2, 4, device="cuda")
    view = pool[:, 1]
    gdn.reorder_states([view, out[:, :1].repeat(3, 1, 1, 1)], torch.zeros(2, 3, **PARENTS))
    assert view._version == pool._version == 1


def test_a_state_saved_for_backward_and_then_moved_is_noticed():
    a = step_args("cuda")
    w = torch.ones(4, 64, 64, device="cuda", requires_grad=True)
    y = (a["state"] * w).sum()
    with torch.no_grad():
        gdn.recurrent_gated_delta_rule(**a)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inference_tensors():
    with torch.inference_mode():
        a = step_args("cuda")
        gdn.recurrent_gated_delta_rule(**a)
    gdn.recurrent_gated_delta_rule(**a)  # they have no versions
    with torch.inference_mode():
        x = torch.arange(6.0, device="cuda").view(6, 1)
    gdn.reorder_states(x, torch.tensor([[1, 1, 1], [0, 0, 0]], **PARENTS))
    assert x.flatten().tolist() == [1, 1, 1, 3, 3, 3]

"""A NaN or an infinity in one drafted token, or in the state, reaches what its path reaches and nothing else: the same
outputs are finite as in the recurrence walked down every path in 64 bits, and these are as close as ever."""
import math

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from parity import BF16_TOL, FP32_TOL
from test_gpu_decode import args, check_o, dev, make, random_parents, tree_reference

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
NAN, INF = math.nan, math.inf


def plant(x, what, t, number):
    """A value that is none into node t of every row (one head of it, one column)."""
    if what == "v":
        x["v"][:, t, -1, 3] = number
    elif what == "whole v":
        x["v"][:, t, -1] = number
    elif what in ("q", "k"):
        x[what][:, t, -1, 7] = number
    elif what == "whole k":
        x["k"][:, t, -1] = number
    elif what in ("g", "beta"):
        x[what][:, t, -1] = number
    elif what == "state":
        x["state"][:, -1, 5, 9] = number


def verify(x, parents, idx=None):
    o = gdn.tree_gated_delta_rule(*args(x), parents.cuda(), x["state"].cuda(), state_indices=x["idx"].cuda()).cpu()
    ref = tree_reference(x, parents, x["state"][x["idx"].long()])
    fine = ref.isfinite()
    assert torch.equal(o.isfinite(), fine), [(~o[..., h, :].isfinite()).sum().item() - (~fine[..., h, :]).sum().item() for h in range(o.shape[2])]
    check_o(torch.where(fine, o, 0), torch.where(fine, ref, 0), x["dtype"], BF16_TOL if x["dtype"] == bf16 else FP32_TOL)
    assert fine.any() and not fine.all()


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("T,K,V", [(7, 128, 128), (20, 64, 64), (33, 128, 64), (48, 64, 128), (64, 128, 128)])
@pytest.mark.parametrize("what,number", [("v", NAN), ("v", INF), ("whole v", -INF), ("k", NAN), ("k", INF), ("whole k", NAN),
                                         ("q", NAN), ("q", INF), ("g", NAN), ("g", INF), ("beta", NAN), ("beta", -INF),
                                         ("state", NAN), ("state", INF)])
def test_tree_a_value_that_is_none(what, number, T, K, V, dtype):
    x = make(2, T, 2, 4, K, V, dtype, seed=51)
    parents = random_parents(2, T, 9)
    parents[0, 1:4] = torch.tensor([0, 0, 1])  # node 1 with a sibling and a child
    plant(x, what, 1, number)
    verify(x, parents)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_tree_several_in_siblings_and_below_a_forgetting_gate(dtype):
    """Several nodes at once, one of them above a gate of -inf, which forgets no NaN; absent nodes that hold more."""
    T = 40
    x = make(2, T, 1, 3, 128, 128, dtype, seed=52)
    parents = random_parents(2, T, 10)
    parents[:, :12] = torch.tensor([-1, 0, 0, 1, 2, 3, 3, 4, -1, 8, 8, -3], dtype=torch.int32)
    parents[:, 20] = 11  # under the absent one
    x["k"][:, 3] = NAN
    x["g"][:, 5] = -INF
    x["v"][0, 7, 1, 100] = INF
    x["q"][1, 9, 0, 0] = NAN
    x["beta"][:, 10, 2] = NAN
    for name in ("q", "k", "v"):
        x[name][:, 11] = NAN
    verify(x, parents)


@pytest.mark.parametrize("T", [9, 30, 40])
def test_tree_values_that_are_none_on_many_heads(T):
    """CTAs that go on to other heads after one with such a value."""
    x = make(40, T, 8, 32, 128, 128, bf16, seed=53)
    parents = random_parents(40, T, 11)
    parents[:, 1:4] = torch.tensor([0, 0, 1], dtype=torch.int32)
    x["v"][::2, 1, 5, 17] = NAN
    x["k"][1::3, 1, 2] = INF
    x["beta"][4, 2, 31] = NAN
    idx, state = x["idx"].cuda(), x["state"].cuda()
    o = gdn.tree_gated_delta_rule(*args(x), parents.cuda(), state, state_indices=idx).cpu()
    some = [0, 1, 3, 4, 25, 38]
    few = {n: (y[some] if isinstance(y, torch.Tensor) and n != "state" else y) for n, y in x.items()}
    ref = tree_reference(few, parents[some], x["state"][x["idx"][some].long()])
    fine = ref.isfinite()
    assert torch.equal(o[some].isfinite(), fine)
    check_o(torch.where(fine, o[some], 0), torch.where(fine, ref, 0), bf16, BF16_TOL)
    assert o[3].isfinite().all() and not o[0].isfinite().all()


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_tree_products_past_the_largest_number(dtype):
    """Finite inputs whose products are infinite: their branch shows it, the others do not."""
    x = make(1, 6, 1, 1, 64, 64, dtype, seed=54)
    parents = torch.tensor([[-1, 0, 1, 0, 3, -1]], dtype=torch.int32)
    x["k"][:, 1:3] *= 3e25
    x["beta"][:, 1:3] = 1.0
    o = gdn.tree_gated_delta_rule(*args(x), parents.cuda(), x["state"].cuda(), state_indices=x["idx"].cuda()).cpu()
    live = [0, 3, 4, 5]
    ref = tree_reference(x, parents, x["state"][x["idx"].long()])
    check_o(o[:, live], ref[:, live], dtype, BF16_TOL if dtype == bf16 else FP32_TOL)

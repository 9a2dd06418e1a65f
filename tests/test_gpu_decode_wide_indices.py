"""64-bit (and unsigned) indices that no 32-bit number holds are out of range or idle, never another slot or token."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from test_gpu_decode import args, check_o, make, reference, tree_reference
from parity import BF16_TOL

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16
UP, DOWN = [2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 33 - 1, 2 ** 62, 2 ** 63 - 1], [-2 ** 31 - 1, -2 ** 32, 1 - 2 ** 32, -2 ** 63]


def test_state_indices():
    n = len(UP) + len(DOWN)
    x = make(n + 1, 2, 1, 2, 64, 64, bf16, seed=41)
    idx = torch.tensor(UP + DOWN + [1], dtype=torch.int64, device="cuda")
    state = x["state"].cuda()
    a = args(x)
    parents = torch.tensor([[-1, 0]] * (n + 1), device="cuda")
    tree = gdn.tree_gated_delta_rule(*a, parents, state, state_indices=idx)
    o = gdn.recurrent_gated_delta_rule(*a, state, state_indices=idx)
    for y in (tree, o):
        assert y[:len(UP)].isnan().all() and (y[len(UP):n] == 0).all() and y[n].isfinite().all()
    keep = [s for s in range(state.shape[0]) if s != 1]
    assert torch.equal(state[keep].cpu(), x["state"][keep])


def test_unsigned_state_indices():
    x = make(3, 1, 1, 2, 64, 64, bf16, seed=42)
    state = x["state"].cuda()
    idx = torch.tensor([2 ** 32 - 1, 2 ** 31, 2], dtype=torch.uint32).cuda()
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=idx)
    assert o[:2].isnan().all() and o[2].isfinite().all()
    wide = torch.tensor([-1, -2 ** 63, 1], dtype=torch.int64).view(torch.uint64).cuda()
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=wide)
    assert o[:2].isnan().all() and o[2].isfinite().all()
    assert torch.equal(state[[0, 3, 4, 5]].cpu(), x["state"][[0, 3, 4, 5]])


def test_token_indices_and_parents():
    wide = UP + DOWN
    x = make(len(wide), 3, 1, 2, 64, 64, bf16, seed=43)
    lists = torch.tensor([[1, w, 0] for w in wide], device="cuda")
    state = x["state"].cuda()
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=x["idx"].cuda(), token_indices=lists)
    h0 = x["state"][x["idx"].long()]
    first, ref_s = reference(x, h0, [[1]] * len(wide))
    for b, w in enumerate(wide):
        check_o(o[b, :1], first[b], bf16)
        slot = int(x["idx"][b])
        if w > 0:
            assert o[b, 1:].isnan().all() and torch.equal(state[slot].cpu(), x["state"][slot])
        else:  # the end of the list
            assert (o[b, 1:] == 0).all() and not torch.equal(state[slot].cpu(), x["state"][slot])
    parents = torch.tensor([[-1, w, 0] for w in wide], device="cuda")
    o = gdn.tree_gated_delta_rule(*args(x), parents, x["state"].cuda(), state_indices=x["idx"].cuda())
    ref = tree_reference(x, torch.tensor([[-1, -2, 0]] * len(wide)), h0)
    check_o(o[:, [0, 2]], ref[:, [0, 2]], bf16, BF16_TOL)
    assert o[:len(UP), 1].isnan().all() and (o[len(UP):, 1] == 0).all()


@pytest.mark.parametrize("wrong", [0, 1, 2])
def test_cu_seqlens(wrong):
    x = make(1, 6, 1, 2, 64, 64, bf16, seed=44, slots=2)
    cu = torch.tensor([0, 3, 6])
    cu[wrong] += 2 ** 32
    state = x["state"].cuda()
    gdn.recurrent_gated_delta_rule(*args(x), state, cu_seqlens=cu.cuda())
    for n in range(2):
        assert torch.equal(state[n].cpu(), x["state"][n]) == (wrong in (n, n + 1))


def test_reorder():
    x = torch.arange(12 * 8, dtype=torch.float32).view(12, 8)
    got = x.cuda()
    parents = torch.tensor([[1, 2 ** 32, 2 ** 31, -2 ** 32, 2 ** 32 - 1, 0]], device="cuda")
    gdn.reorder_states(got, parents)
    got = got.cpu()
    assert torch.equal(got[0], x[1]) and torch.equal(got[5], x[0]) and torch.equal(got[3], x[3])
    assert got[[1, 2, 4]].isnan().all() and torch.equal(got[6:], x[6:])
    got = x.cuda()
    parents = torch.tensor([[1, 1, 1, 3]], dtype=torch.int32, device="cuda")
    idx = torch.tensor([[2 ** 32, 2 ** 32 + 3, 7, 2 ** 63 - 1]], device="cuda")  # beam 1, whom two follow, has no slot
    gdn.reorder_states(got, parents, state_indices=idx)
    got = got.cpu()
    assert got[7].isnan().all()
    assert torch.equal(got[[i for i in range(12) if i != 7]], x[[i for i in range(12) if i != 7]])

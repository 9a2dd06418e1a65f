"""The recurrent step on lists of tokens for many heads, where states come through a ring of slots that two groups of
threads share: rows without a slot, without tokens and with long lists in every order, so that the groups overtake each
other.  Every row is held to the same rows run few at a time, which goes another way, and some to the 64-bit oracle."""
import math

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from parity import FP32_TOL
from test_gpu_decode import args, check_o, check_state, make, reference

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
ROWS, HEADS = 96, 64  # 6144 heads: forty for every SM


def pattern(kind, gen, T):
    """Lists [ROWS, n] and which rows have a slot (0), are idle (1) or name a slot that is none (2)."""
    n = 21
    length = torch.randint(1, 4, (ROWS,), generator=gen)
    off = torch.zeros(ROWS, dtype=torch.long)
    row = torch.arange(ROWS)
    if kind == "every other":
        off = row % 2
    elif kind == "runs":  # several heads of one SM after another, 152 heads apart
        off = (row // 5 % 2) * (1 + row % 2)
    elif kind == "mostly idle":
        off = (torch.rand(ROWS, generator=gen) < 0.9).long()
    elif kind == "long beside short":
        length = torch.where(row % 7 == 3, 20, torch.randint(0, 2, (ROWS,), generator=gen))
    elif kind == "random":
        off = (torch.rand(ROWS, generator=gen) < 0.4).long() * torch.randint(1, 3, (ROWS,), generator=gen)
        length = torch.randint(0, 21, (ROWS,), generator=gen)
    lists = torch.randint(0, T, (ROWS, n), generator=gen)
    lists[torch.arange(n) >= length.unsqueeze(1)] = -1
    return lists.to(torch.int32), off


def check_rows(got, want):
    """Row by row, on the GPU: one wrong state among many is not lost in their mean."""
    err = (got - want).abs().flatten(1).amax(1)
    rms = want.double().square().flatten(1).mean(1).sqrt()
    assert (err <= FP32_TOL * rms).all(), (err / rms).tolist()


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("kind", ["every other", "runs", "mostly idle", "long beside short", "random"])
def test_ring_of_states(kind, with_q, dtype):
    T = 9
    gen = torch.Generator().manual_seed(len(kind))
    x = make(ROWS, T, 16, HEADS, 128, 128, dtype, seed=31, slots=ROWS + 2)
    lists, off = pattern(kind, gen, T)
    idx = torch.where(off == 1, -1, torch.where(off == 2, x["state"].shape[0] + 1, x["idx"].long())).to(torch.int32).cuda()
    lists = lists.cuda()
    a, start = args(x), x["state"].cuda()
    q = a[0] if with_q else None
    want_state, want_o = start.clone(), []
    for b in range(0, ROWS, 16):  # 1024 heads: single warps
        few = slice(b, b + 16)
        o = gdn.recurrent_gated_delta_rule(None if q is None else q[few], *(y[few] for y in a[1:]), want_state,
                                           state_indices=idx[few], token_indices=lists[few])
        want_o.append(o)
    live = [b for b in range(ROWS) if off[b] == 0]
    for trial in range(6):
        state = start.clone()
        o = gdn.recurrent_gated_delta_rule(q, *a[1:], state, state_indices=idx, token_indices=lists)
        untouched = torch.ones(state.shape[0], dtype=torch.bool)
        untouched[x["idx"][live].long()] = False
        assert torch.equal(state[untouched.cuda()], start[untouched.cuda()])
        slots = x["idx"][live].long().cuda()
        check_rows(state[slots], want_state[slots])
        if with_q:
            want = torch.cat(want_o)
            assert torch.equal(o.isnan(), want.isnan())
            assert torch.equal(o[(off == 1).cuda()], want[(off == 1).cuda()])
            check_o(o[live].double(), want[live].double(), dtype)
    for b in live[:3]:
        tokens = [t for t in lists[b].tolist() if t >= 0]
        ref_o, ref_s = reference({n: (y[b:b + 1] if isinstance(y, torch.Tensor) and n != "state" else y) for n, y in x.items()},
                                 x["state"][x["idx"][b:b + 1].long()], [tokens])
        check_state(state[int(x["idx"][b])], ref_s[0])
        if with_q and tokens:
            check_o(o[b, :len(tokens)], ref_o[0], dtype)


def test_ring_shared_slots_into_out_state():
    """Rows that share a slot, through the ring, into states of their own; `state` is only read."""
    gen = torch.Generator().manual_seed(5)
    x = make(ROWS, 5, 16, HEADS, 128, 128, bf16, seed=32, slots=4)
    lists, _ = pattern("random", gen, 5)
    idx = torch.randint(0, 4, (ROWS,), generator=gen).to(torch.int32).cuda()
    a, state, lists = args(x), x["state"].cuda(), lists.cuda()
    out = torch.full((ROWS, HEADS, 128, 128), math.nan, device="cuda")
    gdn.recurrent_gated_delta_rule(None, *a[1:], state, state_indices=idx, token_indices=lists, out_state=out)
    assert torch.equal(state.cpu(), x["state"])
    want = torch.empty_like(out)
    for b in range(0, ROWS, 16):
        few = slice(b, b + 16)
        gdn.recurrent_gated_delta_rule(None, *(y[few] for y in a[1:]), state, state_indices=idx[few],
                                       token_indices=lists[few], out_state=want[few])
    check_rows(out, want)

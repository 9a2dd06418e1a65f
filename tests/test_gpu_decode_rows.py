"""Packed sequences: rows of o that belong to no sequence are 0, whatever the memory held before."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from test_gpu_decode import args, check_o, make, reference

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


def dirty(x):
    """Memory of o's size, given back with something in it."""
    junk = torch.full(x["v"].shape, 7.0, dtype=x["dtype"], device="cuda")
    del junk


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("cu", [[2, 5, 5, 9], [0, 11], [0], [4], [-2, 3, 9, 15], [0, 4, 3, 7], [3, 40]], ids=str)
def test_rows_outside_every_sequence(cu, dtype):
    T = 11
    x = make(1, T, 2, 4, 128, 128, dtype, seed=61, slots=5)
    a, state, offsets = args(x), x["state"].cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda")
    dirty(x)
    o = gdn.recurrent_gated_delta_rule(*a, state, cu_seqlens=offsets)
    claims = torch.zeros(T, dtype=torch.long)  # falling offsets may leave a row to two sequences: then it is either's
    runs = {s: (lo, hi) for s, (lo, hi) in enumerate(zip(cu, cu[1:])) if 0 <= lo <= hi <= T}
    for lo, hi in runs.values():
        claims[lo:hi] += 1
    for s in range(len(cu) - 1):
        if s not in runs:
            assert torch.equal(state[s].cpu(), x["state"][s])
        elif runs[s][0] < runs[s][1]:
            lo, hi = runs[s]
            ref_o, _ = reference(x, x["state"][s:s + 1], [list(range(lo, hi))])
            once = claims[lo:hi] == 1
            check_o(o[0, lo:hi][once.cuda()], ref_o[0][once], dtype)
    assert (o[0, claims == 0] == 0).all()

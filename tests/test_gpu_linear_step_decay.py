"""The step of linear attention at the ends of its decay, against the recurrence in 64 bits."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from parity import FP32_TOL, check
from test_gpu_linear_step import call, make, run

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("size", [1.0, 1e6])
@pytest.mark.parametrize("dtype,T,lists", [(bf16, 1, False), (bf16, 7, False), (f32, 9, False), (bf16, 6, True)])
def test_ends_of_the_decay(dtype, T, lists, size):
    """Heads that keep nothing, almost nothing, a third, almost everything and everything, each by itself."""
    B = 40 if lists else 3  # enough heads for the ring of states
    Hv = 48 if lists else 6
    x = make(B, T, Hv, Hv, 128, 128, dtype, seed=T)
    x["g"] = torch.tensor([-float("inf"), -60.0, -1.0, -1e-3, -1e-6, 0.0]).repeat(Hv // 6)
    x["state"] *= size
    state = x["state"].cuda()
    kw = dict(token_indices=torch.arange(T, dtype=torch.int32).repeat(B, 1).cuda()) if lists else {}
    o = call(x, state, state_indices=x["idx"].cuda(), **kw)
    for b in range(0, B, 7):
        slot = int(x["idx"][b])
        ref_o, ref_s = run(x, b, range(T), x["state"][slot])
        for h in range(6):
            check("state", state[slot, h], ref_s[h], f32, f32, tol=FP32_TOL)
            for t in range(T):
                check("o", o[b, t, h], ref_o[t, h], f32, dtype, tol=FP32_TOL)


@pytest.mark.parametrize("lists", [False, True])
def test_slow_decay_over_many_tokens(lists):
    """4096 tokens on heads that forget 1e-6, 2.9e-8, 5e-4 and 1.1e-3 a token, whose decays fp32 rounds by up to half a step: the
    decay has to be what g says, not what e^g rounds to.

    What an element may be off by: each token rounds the state once to 24 bits, by ulp / sqrt(12) on average, independently,
    for its additions are random; |S| stays below 512, whose ulp is 2^-15, so that six standard deviations of 4096 roundings
    are 6 * 2^-15 / sqrt(12) * 64 = 3.4e-3 (the product and the sum below it round at the size of k v, ulp 2^-20 or less:
    a 32nd of that).  A head that forgets 1.1e-3 may round twice a token, but keeps no more than 1 / (2 * 1.1e-3) = 450 tokens'
    roundings.  A decay that is off by 1.3e-8 or 2.9e-8 a token moves an initial element of 250 by 1.4e-2 or 3e-2."""
    T, Hv = 4096, 64 if lists else 4
    B = 40 if lists else 1
    gen = torch.Generator().manual_seed(8)
    K = V = 128 if lists else 64  # lists: the ring of states takes 128 x 128 alone
    rows = torch.randn(1, T, 2 * K + Hv * V, generator=gen)
    x = dict(q=rows[..., :K].view(1, T, 1, K), k=rows[..., K:2 * K].view(1, T, 1, K), v=rows[..., 2 * K:].view(1, T, Hv, V))
    x["g"] = torch.tensor([-1e-6, -2.9e-8, -5e-4, -1.1e-3]).repeat(Hv // 4)
    first = 64 * torch.randn(1, Hv, K, V, generator=gen)
    state = first.expand(B, -1, -1, -1).contiguous().cuda()
    side = [x[n].expand(B, -1, -1, -1).cuda() for n in ("q", "k", "v")]
    kw = dict(token_indices=torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)) if lists else {}
    gdn.recurrent_linear_attention(None, side[1], side[2], x["g"].cuda(), state, **kw)
    decay = torch.exp(x["g"][:4].double()).cuda()[:, None, None]
    S, k, v = first[0, :4].double().cuda(), x["k"][0, :, 0].double().cuda(), x["v"][0, :, :4].double().cuda()
    for t in range(T):
        S = decay * S + k[t][None, :, None] * v[t][:, None]
    assert S.abs().max() < 512
    assert (state[-1, :4].double() - S).abs().max() < 3.5e-3

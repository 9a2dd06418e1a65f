"""The step of linear attention on a pool of states against the recurrence in 64 bits: slots, packed tokens, lists, states
out of place.  Tolerances as in test_gpu_decode.py: states 1e-5 * RMS, o its rounding on top of that."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from parity import FP32_TOL, check

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


def make(B, T, Hq, Hv, K, V, dtype, seed, slots=None):
    gen = torch.Generator().manual_seed(seed)
    nq = Hq * K
    rows = torch.randn(B, T, 2 * nq + Hv * V, generator=gen).to(dtype)
    x = dict(q=rows[..., :nq].view(B, T, Hq, K), k=rows[..., nq:2 * nq].view(B, T, Hq, K), v=rows[..., 2 * nq:].view(B, T, Hv, V))
    x["g"] = -torch.exp2(-8 * torch.rand(Hv, generator=gen))
    slots = B + 3 if slots is None else slots
    x["state"] = torch.randn(slots, Hv, K, V, generator=gen)
    x["idx"] = torch.randperm(slots, generator=gen)[:B].to(torch.int32)
    return x


def run(x, b, tokens, S):
    """(o [len, Hv, V], state) of row b from S through the tokens; 64 bits."""
    G = x["v"].shape[2] // x["q"].shape[2]
    q, k, v = (x[n][b].double() for n in ("q", "k", "v"))
    decay, S, os = torch.exp(x["g"].double())[:, None, None], S.double(), []
    for t in tokens:
        S = decay * S + k[t].repeat_interleave(G, 0)[:, :, None] * v[t][:, None]
        os.append((S * q[t].repeat_interleave(G, 0)[:, :, None]).sum(1) * q.shape[-1] ** -0.5)
    return torch.stack(os) if os else torch.zeros(0, v.shape[1], v.shape[2]), S


def call(x, state, **kw):
    base = torch.cat([x["q"].flatten(2), x["k"].flatten(2), x["v"].flatten(2)], -1).cuda()
    B, T, Hq, K = x["q"].shape
    nq = Hq * K
    q, k, v = base[..., :nq].view(B, T, Hq, K), base[..., nq:2 * nq].view(B, T, Hq, K), base[..., 2 * nq:].view(x["v"].shape)
    if kw.pop("no_q", False):
        q = None
    return gdn.recurrent_linear_attention(q, k, v, x["g"].cuda(), state, **kw)


CASES = [(1, 1, 16, 32, 128, 128, bf16), (5, 1, 2, 8, 128, 128, bf16), (3, 1, 1, 1, 64, 64, f32), (2, 7, 2, 6, 128, 64, bf16),
         (4, 8, 4, 4, 64, 128, bf16), (3, 9, 2, 4, 128, 128, f32), (2, 100, 1, 2, 128, 128, bf16)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_step(case):
    x = make(*case, seed=sum(case[:6]))
    state = x["state"].cuda()
    o = call(x, state, state_indices=x["idx"].cuda())
    left = torch.ones(state.shape[0], dtype=torch.bool)
    for b in range(case[0]):
        slot = int(x["idx"][b])
        left[slot] = False
        ref_o, ref_s = run(x, b, range(case[1]), x["state"][slot])
        check("o", o[b], ref_o, f32, case[6], tol=FP32_TOL)
        check("state", state[slot], ref_s, f32, f32, tol=FP32_TOL)
    assert torch.equal(state.cpu()[left], x["state"][left])


@pytest.mark.parametrize("B,Hv", [(6, 4), (48, 64)])  # few heads, and enough for the ring of states
@pytest.mark.parametrize("with_q", [False, True])
def test_lists_idle_rows_and_bad_tokens(B, Hv, with_q):
    x = make(B, 6, 2, Hv, 128, 128, bf16, seed=B)
    lists = torch.full((B, 6), -1, dtype=torch.int32)
    for b in range(B):
        n = b % 7
        lists[b, :n] = torch.arange(n, dtype=torch.int32).flip(0)
    lists[5, 1] = 17  # no such token
    idx = x["idx"].clone()
    idx[2] = -1
    state = x["state"].cuda()
    o = call(x, state, state_indices=idx.cuda(), token_indices=lists.cuda(), no_q=not with_q)
    assert (o is None) == (not with_q)
    for b in range(B):
        slot, tokens = int(x["idx"][b]), [t for t in lists[b].tolist() if t >= 0]
        if b in (2, 5):  # idle, and one whose list names no token: the slot stays
            assert torch.equal(state[slot].cpu(), x["state"][slot])
            continue
        ref_o, ref_s = run(x, b, tokens, x["state"][slot])
        check("state", state[slot], ref_s, f32, f32, tol=FP32_TOL)
        if with_q:
            if tokens:
                check("o", o[b, :len(tokens)], ref_o, f32, bf16, tol=FP32_TOL)
            assert (o[b, len(tokens):] == 0).all()
    if with_q:
        assert (o[2] == 0).all() and o[5, 1:].isnan().all()


def test_packed_tokens_and_states_out_of_place():
    lens = [1, 4, 0, 12, 3]
    x = make(1, sum(lens) + 2, 2, 4, 64, 128, bf16, seed=6, slots=9)
    cu = torch.tensor([0, 1, 5, 5, 17, 20], dtype=torch.int32)
    idx = torch.tensor([8, 0, 3, 0, 1], dtype=torch.int32)  # two rows continue one state
    state, out = x["state"].cuda(), torch.full((5, 4, 64, 128), 7.0, device="cuda")
    o = call(x, state, state_indices=idx.cuda(), cu_seqlens=cu.cuda(), out_state=out)
    assert torch.equal(state.cpu(), x["state"]) and (o[0, 20:] == 0).all()
    for s, n in enumerate(lens):
        ref_o, ref_s = run(x, 0, range(int(cu[s]), int(cu[s + 1])), x["state"][int(idx[s])])
        check("state", out[s], ref_s, f32, f32, tol=FP32_TOL)
        if n:
            check("o", o[0, int(cu[s]):int(cu[s + 1])], ref_o, f32, bf16, tol=FP32_TOL)


def test_without_decay_it_is_the_sum_of_products():
    x = make(2, 3, 1, 2, 64, 64, f32, seed=1)
    x["g"] = torch.zeros(2)
    a, b = x["state"].cuda(), x["state"].cuda()
    o = call(x, a, state_indices=x["idx"].cuda())
    side = [x[n].cuda() for n in ("q", "k", "v")]
    assert torch.equal(gdn.recurrent_linear_attention(*side, None, b, state_indices=x["idx"].cuda()), o) and torch.equal(a, b)


def test_graph():
    x = make(3, 2, 2, 4, 128, 128, bf16, seed=13)
    idx, first = x["idx"].cuda(), x["state"].cuda()
    side = [x[n].cuda() for n in ("q", "k", "v", "g")]
    gdn.recurrent_linear_attention(*side, first, state_indices=idx)
    two = gdn.recurrent_linear_attention(*side, first, state_indices=idx)
    state = x["state"].cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdn.recurrent_linear_attention(*side, state, state_indices=idx)
    state.copy_(x["state"])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, two) and torch.equal(state, first)

"""The decoding operators on the state pool against 64-bit references: the token-by-token oracle for the
recurrence, the same recurrence walked down every path for trees.

Tolerances are those of ``parity.py``: the states are fp32 sums of at most a few hundred terms whose errors do
not grow along the tokens (every step contracts), so they are held to 1e-5 * RMS with bf16 inputs too; o is held
to its rounding on top of 1e-5 * RMS (recurrence) or 2e-3 * RMS (tree, whose bf16 kernels may split operands)."""
import math

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
import oracle
from parity import BF16_TOL, FP32_TOL, check

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


def make(B, T, Hq, Hv, K, V, dtype, seed=0, slots=None, packed=True):
    """Inputs on the CPU; q, k, v as views of one row per token, as one projection writes them."""
    gen = torch.Generator().manual_seed(seed)
    nq = Hq * K
    rows = torch.empty(B, T, 2 * nq + Hv * V, dtype=dtype)
    q, k, v = rows[..., :nq].view(B, T, Hq, K), rows[..., nq:2 * nq].view(B, T, Hq, K), rows[..., 2 * nq:].view(B, T, Hv, V)
    for x in (q, k):
        y = torch.randn(B, T, Hq, K, generator=gen)
        x.copy_(y / y.norm(dim=-1, keepdim=True))
    v.copy_(torch.randn(B, T, Hv, V, generator=gen))
    if not packed:
        q, k, v = (x.contiguous() for x in (q, k, v))
    g = -torch.nn.functional.softplus(torch.randn(B, T, Hv, generator=gen))
    beta = torch.sigmoid(torch.randn(B, T, Hv, generator=gen))
    slots = B + 3 if slots is None else slots
    state = 0.1 * torch.randn(slots, Hv, K, V, generator=gen)
    idx = torch.randperm(slots, generator=gen)[:B].to(torch.int32)
    return dict(q=q, k=k, v=v, g=g, beta=beta, state=state, idx=idx, dtype=dtype, scale=K ** -0.5)


def dev(t):
    """To the GPU, strides and all."""
    if t is None or t.is_contiguous():
        return None if t is None else t.cuda()
    base = t._base if t._base is not None else t
    return base.cuda().as_strided(t.shape, t.stride(), t.storage_offset())


def args(x):
    return [dev(x[n]) for n in ("q", "k", "v", "g", "beta")]


def reference(x, h0, tokens=None):
    """(o, final states) of the rows from h0 [B, Hv, K, V], through `tokens` of each row where given."""
    q, k, v, g, beta = (x[n] for n in ("q", "k", "v", "g", "beta"))
    if tokens is None:
        return oracle.oracle_fwd(q.contiguous(), k.contiguous(), v.contiguous(), g, beta, x["scale"], h0)
    os, hs = [], []
    for b, t in enumerate(tokens):
        if len(t) == 0:
            os.append(torch.zeros(0, v.shape[2], v.shape[3], dtype=torch.float64))
            hs.append(h0[b].double())
            continue
        o, h = oracle.oracle_fwd(*(y[b:b + 1, t].contiguous() for y in (q, k, v, g, beta)), x["scale"], h0[b:b + 1].contiguous())
        os.append(torch.as_tensor(o)[0])
        hs.append(torch.as_tensor(h)[0])
    return os, torch.stack(hs)


def check_state(got, ref):
    check("state", got, ref, f32, f32, tol=FP32_TOL)


def check_o(got, ref, dtype, tol=FP32_TOL):
    check("o", got, ref, f32, dtype, tol=tol)


STEP_CASES = [  # B, T, Hq, Hv, K, V, dtype
    (1, 1, 16, 32, 128, 128, bf16), (5, 1, 2, 8, 128, 128, bf16), (3, 1, 1, 1, 64, 64, f32),
    (2, 7, 2, 6, 128, 64, bf16), (4, 8, 4, 4, 64, 128, bf16), (3, 9, 2, 4, 128, 128, f32),
    (1, 17, 1, 3, 64, 64, bf16), (2, 300, 1, 2, 128, 128, bf16), (1, 65, 2, 2, 128, 128, f32),
    (40, 2, 4, 16, 128, 128, bf16),
]


@pytest.mark.parametrize("case", STEP_CASES, ids=str)
def test_recurrent(case):
    x = make(*case, seed=sum(case[:6]))
    state = x["state"].cuda()
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=x["idx"].cuda())
    ref_o, ref_s = reference(x, x["state"][x["idx"].long()])
    assert o.dtype == x["dtype"]
    check_o(o, ref_o, x["dtype"])
    check_state(state[x["idx"].long().cuda()], ref_s)
    rest = torch.ones(state.shape[0], dtype=torch.bool)
    rest[x["idx"].long()] = False
    assert torch.equal(state.cpu()[rest], x["state"][rest])


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_recurrent_continues_a_prefill(dtype):
    """Prefill through the chunked operator, then tokens one by one: the same as one prefill over all."""
    x = make(2, 75, 2, 4, 128, 128, dtype, seed=3, packed=False)
    q, k, v, g, beta = args(x)
    cut = 70
    _, state = gdn.chunk_gated_delta_rule(q[:, :cut], k[:, :cut], v[:, :cut], g[:, :cut], beta[:, :cut], output_final_state=True)
    outs = [gdn.recurrent_gated_delta_rule(*(y[:, t:t + 1] for y in (q, k, v, g, beta)), state) for t in range(cut, 75)]
    ref_o, ref_s = oracle.oracle_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["scale"], None)
    tol = FP32_TOL if dtype == f32 else BF16_TOL
    check("o", torch.cat(outs, 1), torch.as_tensor(ref_o)[:, cut:], dtype, dtype, tol=tol)
    check("state", state, ref_s, dtype, f32, tol=tol)


def test_recurrent_idle_rows_and_slots_out_of_range():
    x = make(5, 3, 2, 4, 128, 128, bf16, seed=4)
    state = x["state"].cuda()
    idx = x["idx"].clone()
    idx[1], idx[3] = -1, state.shape[0]
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=idx.cuda())
    keep = [0, 2, 4]
    ref_o, ref_s = reference(x, x["state"][x["idx"].long()])
    check_o(o[keep], torch.as_tensor(ref_o)[keep], bf16)
    assert (o[1] == 0).all() and o[3].isnan().all()
    expect = x["state"].clone()
    assert torch.equal(state.cpu()[x["idx"][[1, 3]].long()], expect[x["idx"][[1, 3]].long()])
    check_state(state[x["idx"][keep].long().cuda()], torch.as_tensor(ref_s)[keep])


@pytest.mark.parametrize("with_q", [True, False])
def test_recurrent_token_lists(with_q):
    """Rows of different lengths, an empty one, tokens out of order, and one list with an index that is none."""
    x = make(6, 9, 2, 6, 128, 128, bf16, seed=5)
    lists = [[0, 3, 4], [], list(range(9)), [8, 2, 2], [5], [1, 9, 2]]
    idxs = torch.full((6, 10), -1, dtype=torch.int32)
    for b, t in enumerate(lists):
        idxs[b, :len(t)] = torch.tensor(t, dtype=torch.int32)
    idxs[0, 5] = 7  # past the end of the list: not read as a token
    state = x["state"].cuda()
    a = args(x)
    o = gdn.recurrent_gated_delta_rule(a[0] if with_q else None, *a[1:], state, state_indices=x["idx"].cuda(),
                                       token_indices=idxs.cuda())
    good = lists[:5]
    ref_o, ref_s = reference(x, x["state"][x["idx"].long()], good)
    check_state(state[x["idx"][:5].long().cuda()], ref_s)
    assert torch.equal(state.cpu()[int(x["idx"][5])], x["state"][int(x["idx"][5])])
    if not with_q:
        assert o is None
        return
    assert o.shape == (6, 10, 6, 128)
    for b, t in enumerate(good):
        if t:
            check_o(o[b, :len(t)], ref_o[b], bf16)
        assert (o[b, len(t):] == 0).all()
    first, _ = reference(x, x["state"][x["idx"].long()], lists[:5] + [[1]])
    check_o(o[5, :1], first[5], bf16)
    assert o[5, 1:].isnan().all()


def test_recurrent_varlen():
    lens = [1, 4, 0, 12, 3]
    x = make(1, sum(lens) + 2, 2, 4, 64, 128, bf16, seed=6, slots=9)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    idx = torch.tensor([8, 0, 3, 5, 1], dtype=torch.int32)
    state = x["state"].cuda()
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=idx.cuda(), cu_seqlens=cu.cuda())
    assert o.shape == x["v"].shape
    for s, n in enumerate(lens):
        lo = int(cu[s])
        if n == 0:
            assert torch.equal(state[3].cpu(), x["state"][3])
            continue
        ref_o, ref_s = reference(x, x["state"][idx[s:s + 1].long()], [list(range(lo, lo + n))])
        check_o(o[0, lo:lo + n], ref_o[0], bf16)
        check_state(state[int(idx[s])], ref_s[0])


def test_recurrent_varlen_offsets_out_of_range_touch_nothing():
    x = make(1, 6, 1, 2, 64, 64, f32, seed=7, slots=3)
    cu = torch.tensor([-2, 3, 9, 5], dtype=torch.int32)
    state = x["state"].cuda()
    gdn.recurrent_gated_delta_rule(*args(x), state, cu_seqlens=cu.cuda())
    assert torch.equal(state.cpu(), x["state"])


def test_recurrent_out_state_with_shared_slots():
    """Beams that continue one parent read the same slot and write their own."""
    x = make(4, 2, 2, 4, 128, 128, bf16, seed=8)
    idx = torch.tensor([2, 2, 5, -1], dtype=torch.int32)
    state = x["state"].cuda()
    out = torch.full((4, 4, 128, 128), 7.0, device="cuda")
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=idx.cuda(), out_state=out)
    ref_o, ref_s = reference(x, x["state"][idx.clamp(min=0).long()])
    check_o(o[:3], torch.as_tensor(ref_o)[:3], bf16)
    check_state(out[:3], torch.as_tensor(ref_s)[:3])
    assert (o[3] == 0).all() and (out[3] == 7).all()
    assert torch.equal(state.cpu(), x["state"])


def test_recurrent_gates_at_their_ends():
    """g = -inf forgets the state, g = 0 keeps it, beta = 0 writes nothing, beta = 1 all of it."""
    x = make(2, 4, 1, 4, 128, 128, f32, seed=9)
    x["g"][:, 1, 0] = -math.inf
    x["g"][:, :, 1] = 0.0
    x["beta"][:, :, 2] = 0.0
    x["beta"][:, :, 3] = 1.0
    state = x["state"].cuda()
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=x["idx"].cuda())
    ref_o, ref_s = reference(x, x["state"][x["idx"].long()])
    check_o(o, ref_o, f32)
    check_state(state[x["idx"].long().cuda()], ref_s)


def test_recurrent_layouts():
    """Views with every order of batch, token and head, reversed widths (copied), int64 indices, a strided pool."""
    x = make(3, 4, 2, 4, 128, 64, bf16, seed=10, packed=False)
    pool = torch.zeros(x["state"].shape[0], 2, *x["state"].shape[1:], device="cuda")
    pool[:, 1] = x["state"].cuda()
    state = pool[:, 1]
    q = x["q"].cuda().permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    k = x["k"].cuda().transpose(-1, -2).contiguous().transpose(-1, -2)
    v = torch.zeros(3, 4, 4, 67, dtype=bf16, device="cuda")[..., 3:]
    v.copy_(x["v"])
    g = x["g"].cuda().transpose(0, 2).contiguous().transpose(0, 2)
    beta = x["beta"].cuda().double()
    o = gdn.recurrent_gated_delta_rule(q, k, v, g, beta, state, state_indices=x["idx"].cuda().long())
    ref_o, ref_s = reference(x, x["state"][x["idx"].long()])
    check_o(o, ref_o, bf16)
    check_state(state[x["idx"].long().cuda()], ref_s)
    assert (pool[:, 0] == 0).all()


def test_recurrent_empty():
    x = make(2, 0, 1, 2, 64, 64, bf16, seed=11)
    state = x["state"].cuda()
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=x["idx"].cuda())
    assert o.shape == (2, 0, 2, 64) and torch.equal(state.cpu(), x["state"])
    out = torch.empty(2, 2, 64, 64, device="cuda")
    gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=x["idx"].cuda(), out_state=out)
    assert torch.equal(out.cpu(), x["state"][x["idx"].long()])
    x = make(0, 3, 1, 2, 64, 64, bf16, seed=11)
    o = gdn.recurrent_gated_delta_rule(*args(x), state)
    assert o.shape == (0, 3, 2, 64) and torch.equal(state.cpu(), make(2, 0, 1, 2, 64, 64, bf16, seed=11)["state"])


def test_slots_beyond_32_bit_offsets():
    """A pool of over 2^31 floats: the last slot is read and written at its own place."""
    Hv, K, V = 64, 128, 128
    slots = 2 ** 31 // (Hv * K * V) + 2
    x = make(1, 2, 16, Hv, K, V, bf16, seed=12, slots=1)
    state = torch.empty(slots, Hv, K, V, device="cuda")
    state[0], state[slots - 1] = 3.0, x["state"][0].cuda()
    idx = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    par = torch.tensor([[-1, 0]], dtype=torch.int32, device="cuda")
    tree_o = gdn.tree_gated_delta_rule(*args(x), par, state, state_indices=idx)
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=idx)
    ref_o, ref_s = reference(x, x["state"])
    check_o(o, ref_o, bf16)
    check_o(tree_o, ref_o, bf16, tol=BF16_TOL)
    check_state(state[slots - 1], torch.as_tensor(ref_s)[0])
    assert (state[0] == 3.0).all()
    gdn.reorder_states(state, torch.tensor([[1, 1]], device="cuda"),
                       state_indices=torch.tensor([[0, slots - 1]], device="cuda"))
    assert torch.equal(state[0], state[slots - 1])


def test_side_stream_and_graph():
    x = make(3, 2, 2, 4, 128, 128, bf16, seed=13)
    a, idx = args(x), x["idx"].cuda()
    par = torch.tensor([[-1, 0]] * 3, dtype=torch.int32, device="cuda")
    first = x["state"].cuda()
    one = gdn.recurrent_gated_delta_rule(*a, first, state_indices=idx)
    two = gdn.recurrent_gated_delta_rule(*a, first, state_indices=idx)
    t_two = gdn.tree_gated_delta_rule(*a, par, first, state_indices=idx)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    state = x["state"].cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = gdn.recurrent_gated_delta_rule(*a, state, state_indices=idx)
    side.synchronize()
    assert torch.equal(got, one)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdn.recurrent_gated_delta_rule(*a, state, state_indices=idx)
        t = gdn.tree_gated_delta_rule(*a, par, state, state_indices=idx)
    state.copy_(x["state"])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, two) and torch.equal(state, first) and torch.equal(t, t_two)


# ---- trees ----------------------------------------------------------------------------------------


def tree_reference(x, parents, h0):
    """The recurrence walked down every path in 64 bits; absent nodes give 0."""
    B, T, Hv = x["g"].shape
    G = Hv // x["q"].shape[2]
    q, k = (x[n].double().repeat_interleave(G, 2) for n in ("q", "k"))
    v, g, beta = (x[n].double() for n in ("v", "g", "beta"))
    o = torch.zeros(v.shape, dtype=torch.float64)
    for b in range(B):
        after = {-1: h0[b].double()}
        for t in range(T):
            p = int(parents[b, t])
            if p not in after:  # absent, or under such a node
                continue
            S = after[p] * torch.exp(g[b, t])[:, None, None]
            d = beta[b, t][:, None] * (v[b, t] - torch.einsum("hkv,hk->hv", S, k[b, t]))
            S = S + torch.einsum("hk,hv->hkv", k[b, t], d)
            after[t] = S
            o[b, t] = x["scale"] * torch.einsum("hkv,hk->hv", S, q[b, t])
    return o


def random_parents(B, T, seed):
    gen = torch.Generator().manual_seed(seed)
    return ((torch.rand(B, T, generator=gen) * (torch.arange(T) + 1)).long() - 1).to(torch.int32)


TREE_CASES = [  # B, T, Hq, Hv, K, V, dtype
    (1, 1, 16, 32, 128, 128, bf16), (2, 7, 2, 8, 128, 128, bf16), (3, 16, 1, 2, 64, 64, f32),
    (2, 17, 2, 6, 128, 64, bf16), (2, 33, 2, 2, 64, 128, bf16), (2, 64, 1, 4, 128, 128, bf16),
    (1, 64, 2, 2, 128, 128, f32), (2, 31, 1, 1, 64, 64, bf16), (9, 48, 2, 4, 128, 128, bf16), (1, 50, 1, 3, 128, 64, f32),
]


@pytest.mark.parametrize("case", TREE_CASES, ids=str)
def test_tree(case):
    x = make(*case, seed=sum(case[:6]) + 1)
    parents = random_parents(case[0], case[1], 1)
    state = x["state"].cuda()
    o = gdn.tree_gated_delta_rule(*args(x), parents.cuda(), state, state_indices=x["idx"].cuda())
    check_o(o, tree_reference(x, parents, x["state"][x["idx"].long()]), x["dtype"], BF16_TOL if x["dtype"] == bf16 else FP32_TOL)
    assert torch.equal(state.cpu(), x["state"])


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("shape", ["chain", "star", "absent"])
def test_tree_shapes(shape, dtype):
    """A chain without decay and with full writes (the corrections then reach furthest), children of the state
    only, and absent nodes with children."""
    B, T = 2, 64
    x = make(B, T, 1, 2, 128, 128, dtype, seed=21)
    if shape == "chain":
        parents = (torch.arange(T) - 1).expand(B, T).to(torch.int32)
        x["g"][:] = 0.0
        x["beta"][:] = 1.0
    elif shape == "star":
        parents = torch.full((B, T), -1, dtype=torch.int32)
    else:
        parents = random_parents(B, T, 2)
        parents[:, 5], parents[:, 11], parents[1, 0] = -2, -7, -2
        parents[:, 12], parents[:, 40] = 11, 12
        for name in ("q", "k", "v", "g", "beta"):  # what an absent node holds reaches nobody
            x[name][:, [5, 11]] = math.nan
            x[name][1, 0] = math.inf
    state = x["state"].cuda()
    o = gdn.tree_gated_delta_rule(*args(x), parents.cuda(), state, state_indices=x["idx"].cuda())
    ref = tree_reference(x, parents, x["state"][x["idx"].long()])
    check_o(o, ref, dtype, BF16_TOL if dtype == bf16 else FP32_TOL)
    if shape == "absent":
        assert (o[:, [5, 11, 12, 40]] == 0).all() and (o[1, 0] == 0).all()


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_tree_bad_parents_idle_rows(dtype):
    x = make(4, 20, 2, 4, 128, 128, dtype, seed=22)
    parents = random_parents(4, 20, 3)
    bad = parents.clone()
    bad[0, 6], bad[0, 7], bad[0, 8] = 6, 100, 7  # itself, far outside, a child of that
    ok = parents.clone()
    ok[0, 6], ok[0, 7], ok[0, 8] = -2, -2, 7
    idx = x["idx"].clone()
    idx[1], idx[2] = -3, x["state"].shape[0] + 5
    state = x["state"].cuda()
    o = gdn.tree_gated_delta_rule(*args(x), bad.cuda(), state, state_indices=idx.cuda())
    ref = tree_reference(x, ok, x["state"][x["idx"].long()])
    under = {6, 7, 8}
    for t in range(20):
        if int(ok[0, t]) in under:
            under.add(t)
    under = sorted(under)
    live = [t for t in range(20) if t not in under]
    assert o[0, under].isnan().all() and (o[1] == 0).all() and o[2].isnan().all()
    tol = BF16_TOL if dtype == bf16 else FP32_TOL
    check_o(o[0, live], ref[0, live], dtype, tol)
    check_o(o[3], ref[3], dtype, tol)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_tree_gates_at_their_ends(dtype):
    x = make(2, 24, 1, 3, 128, 128, dtype, seed=23)
    x["g"][:, 3] = -math.inf
    x["g"][:, 4, 1] = -200.0
    x["beta"][:, 5] = 0.0
    parents = random_parents(2, 24, 4)
    parents[:, 4] = 3
    o = gdn.tree_gated_delta_rule(*args(x), parents.cuda(), x["state"].cuda(), state_indices=x["idx"].cuda())
    check_o(o, tree_reference(x, parents, x["state"][x["idx"].long()]), dtype, BF16_TOL if dtype == bf16 else FP32_TOL)


def test_tree_then_accepted_path():
    """Verify a tree, then move the state along one of its paths: the next token sees that path."""
    x = make(3, 12, 2, 4, 128, 128, bf16, seed=24)
    parents = random_parents(3, 12, 5)
    state = x["state"].cuda()
    a, idx = args(x), x["idx"].cuda()
    o = gdn.tree_gated_delta_rule(*a, parents.cuda(), state, state_indices=idx)
    paths, idxs = [], torch.full((3, 12), -1, dtype=torch.int32)
    for b in range(3):
        t, path = 11 - b, []
        while t >= 0:
            path.insert(0, t)
            t = int(parents[b, t])
        paths.append(path)
        idxs[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
    gdn.recurrent_gated_delta_rule(None, *a[1:], state, state_indices=idx, token_indices=idxs.cuda())
    ref_o, ref_s = reference(x, x["state"][x["idx"].long()], paths)
    check_state(state[idx.long()], ref_s)
    for b in range(3):
        check_o(o[b, paths[b]], ref_o[b], bf16, tol=BF16_TOL)


def test_tree_layouts_and_empty():
    x = make(2, 10, 2, 4, 64, 128, bf16, seed=25, packed=False)
    q = x["q"].cuda().permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    k = torch.zeros(2, 10, 2, 65, dtype=bf16, device="cuda")[..., 1:]
    k.copy_(x["k"])
    v = torch.zeros(2, 10, 4, 131, dtype=bf16, device="cuda")[..., :128]
    v.copy_(x["v"])
    parents = random_parents(2, 10, 6)
    o = gdn.tree_gated_delta_rule(q, k, v, x["g"].cuda(), x["beta"].cuda(), parents.cuda().long(), x["state"].cuda(),
                                  state_indices=x["idx"].cuda())
    check_o(o, tree_reference(x, parents, x["state"][x["idx"].long()]), bf16, BF16_TOL)
    e = make(2, 0, 1, 2, 64, 64, bf16)
    assert gdn.tree_gated_delta_rule(*args(e), torch.empty(2, 0, dtype=torch.int32, device="cuda"), e["state"].cuda()).numel() == 0


@pytest.mark.parametrize("T", [5, 40])
def test_tree_many_heads_with_idle_rows(T):
    """More heads than the GPU takes at once, rows without a slot between the others: every CTA's next heads."""
    x = make(30, T, 8, 32, 128, 128, bf16, seed=26)
    parents = random_parents(30, T, 7)
    idx = x["idx"].clone()
    idx[3::4], idx[5] = -1, x["state"].shape[0]
    o = gdn.tree_gated_delta_rule(*args(x), parents.cuda(), x["state"].cuda(), state_indices=idx.cuda())
    some = [0, 1, 13, 28]
    few = {n: (y[some] if isinstance(y, torch.Tensor) and n != "state" else y) for n, y in x.items()}
    ref = tree_reference(few, parents[some], x["state"][x["idx"][some].long()])
    check_o(o[some], ref, bf16, BF16_TOL)
    assert (o[3::4] == 0).all() and o[5].isnan().all()
    live = [b for b in range(30) if b % 4 != 3 and b != 5]
    assert o[live].isfinite().all() and (o[live].float().abs().amax(dim=(1, 3)) > 0).all()


def test_tree_many_heads_ahead():
    """The widest trees whose next state is asked for while a head's products run."""
    test_tree_many_heads_with_idle_rows(32)


def test_recurrent_many_heads_with_idle_rows():
    x = make(50, 3, 8, 32, 128, 128, bf16, seed=27)
    idx = x["idx"].clone()
    idx[3::4], idx[5] = -1, x["state"].shape[0]
    lists = torch.tensor([[2, 0, -1], [1, -1, 0], [0, 1, 2], [-1, -1, -1], [0, 3, 1]], dtype=torch.int32).repeat(10, 1)
    state = x["state"].cuda()
    o = gdn.recurrent_gated_delta_rule(*args(x), state, state_indices=idx.cuda(), token_indices=lists.cuda())
    before = x["state"][x["idx"].long()]
    for b in (0, 1, 2, 4, 17, 32, 49):
        tokens = [t for t in lists[b].tolist()]
        tokens = tokens[:tokens.index(-1)] if -1 in tokens else tokens
        bad = 3 in tokens
        if b == 4 or bad:
            assert bad and o[b, 1:].isnan().all()
            assert torch.equal(state[int(x["idx"][b])].cpu(), before[b])
            continue
        ref_o, ref_s = reference({n: (y[b:b + 1] if isinstance(y, torch.Tensor) and n != "state" else y) for n, y in x.items()},
                                 before[b:b + 1], [tokens])
        check_state(state[int(x["idx"][b])], ref_s[0])
        check_o(o[b, :len(tokens)], ref_o[0], bf16)
        assert (o[b, len(tokens):] == 0).all()
    assert (o[3::4] == 0).all() and o[5].isnan().all()
    for b in (3, 5, 7):
        assert torch.equal(state[int(x["idx"][b])].cpu(), before[b])


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("with_q", [True, False])
def test_recurrent_token_lists_many_heads(with_q, dtype):
    """Lists on more heads than the GPU takes at once, some longer than what is fetched ahead, an empty and an idle row
    and one whose list holds an index that is none."""
    x = make(30, 12, 16, 64, 128, 128, dtype, seed=29, slots=31)
    gen = torch.Generator().manual_seed(3)
    idxs, lists = torch.full((30, 11), -1, dtype=torch.int32), []
    for b in range(30):
        n = int(torch.randint(0, 12, (1,), generator=gen))
        lists.append(torch.randint(0, 12, (n,), generator=gen).tolist())
        idxs[b, :n] = torch.tensor(lists[b], dtype=torch.int32)
    lists[4], idxs[4, 0] = [], -1
    idxs[9, :3], lists[9] = torch.tensor([3, 12, 1], dtype=torch.int32), [3]
    idx = x["idx"].clone()
    idx[20], lists[20] = -1, []
    state, a = x["state"].cuda(), args(x)
    o = gdn.recurrent_gated_delta_rule(a[0] if with_q else None, *a[1:], state, state_indices=idx.cuda(),
                                       token_indices=idxs.cuda())
    h0 = x["state"][x["idx"].long()]
    ref_o, ref_s = reference(x, h0, lists)
    ref_s[9] = h0[9]
    check_state(state[x["idx"].long().cuda()], ref_s)
    if not with_q:
        assert o is None
        return
    for b, t in enumerate(lists):
        if t:
            check_o(o[b, :len(t)], ref_o[b], dtype)
        assert o[b, len(t):].isnan().all() if b == 9 else (o[b, len(t):] == 0).all()


@pytest.mark.parametrize("layout", ["heads outside", "padded rows", "tokens outside", "one shared row", "odd offset"])
@pytest.mark.parametrize("op", ["tree", "recurrent"])
def test_layouts(layout, op):
    """Views that a tensor map can describe, that can only be copied in 16-byte pieces, and that cannot even be that."""
    x = make(40, 6, 4, 8, 128, 128, bf16, seed=28, packed=False)

    def view(t):
        if layout == "heads outside":
            return t.cuda().transpose(1, 2).contiguous().transpose(1, 2)
        if layout == "tokens outside":
            return t.cuda().transpose(0, 1).contiguous().transpose(0, 1)
        if layout == "padded rows":
            wide = torch.zeros(*t.shape[:2], t.shape[2] * t.shape[3] + 24, dtype=t.dtype, device="cuda")
            v = wide[..., 8:8 + t.shape[2] * t.shape[3]].view(t.shape)
        elif layout == "odd offset":
            v = torch.zeros(t.numel() + 3, dtype=t.dtype, device="cuda")[3:].view(t.shape)
        else:  # every batch row is the same memory
            return t[:1].cuda().expand(t.shape)
        v.copy_(t)
        return v

    if layout == "one shared row":
        for n in ("q", "k", "v", "g", "beta"):
            x[n] = x[n][:1].expand(x[n].shape).contiguous()
    a = [view(x[n]) for n in ("q", "k", "v")] + [x["g"].cuda(), x["beta"].cuda()]
    state, idx = x["state"].cuda(), x["idx"].cuda()
    h0 = x["state"][x["idx"].long()]
    if op == "tree":
        parents = random_parents(40, 6, 8)
        o = gdn.tree_gated_delta_rule(*a, parents.cuda(), state, state_indices=idx)
        check_o(o, tree_reference(x, parents, h0), bf16, BF16_TOL)
    else:
        o = gdn.recurrent_gated_delta_rule(*a, state, state_indices=idx)
        ref_o, ref_s = reference(x, h0)
        check_o(o, ref_o, bf16)
        check_state(state[idx.long()], ref_s)

"""Decoding operators of the gated delta rule, at sizes of real use.

Four operators, each as plain torch operations in 32 bits (``own`` false) and as the calls a user
makes of this package (``own`` true), on the same inputs:

* ``step``: a run of new tokens per sequence moves the sequence's state, held in a pool of slots
  (``recurrent_gated_delta_rule``);
* ``tree``: a tree of drafted tokens is answered from a state that stays as it is
  (``tree_gated_delta_rule``);
* ``beam``: one selection of a beam search over beams and vocabulary (``beam_search_step``);
* ``reorder``: the beams' states follow the selection (``reorder_states``).

``own`` is set from outside.
"""
import torch

own = False

_SETTLED = -1  # token of a hypothesis that is carried over unchanged


def listed():
    return [
        # one sequence decoding one token: all that counts is latency
        dict(name="step_one_token", op="step", B=1, T=1, Hq=16, Hv=32, K=128, V=128, dtype="bf16", path=False),
        # a serving batch, one token each
        dict(name="step_batch", op="step", B=64, T=1, Hq=16, Hv=32, K=128, V=128, dtype="bf16", path=False),
        # the accepted paths of drafted trees moved into the states, up to six tokens each; no output wanted
        dict(name="step_accepted_paths", op="step", B=96, T=6, Hq=16, Hv=64, K=128, V=128, dtype="bf16", path=True),
        # 32-bit activations with narrow heads, three tokens at once
        dict(name="step_fp32_narrow", op="step", B=37, T=3, Hq=4, Hv=8, K=64, V=64, dtype="fp32", path=False),
        # a small drafted tree for one sequence
        dict(name="tree_one_sequence", op="tree", B=1, T=7, Hq=16, Hv=32, K=128, V=128, dtype="bf16"),
        # an ordinary verification batch, an odd number of nodes
        dict(name="tree_batch", op="tree", B=16, T=33, Hq=16, Hv=32, K=128, V=128, dtype="bf16"),
        # the widest trees for many sequences and many heads
        dict(name="tree_wide", op="tree", B=64, T=64, Hq=16, Hv=64, K=128, V=128, dtype="bf16"),
        # one request, few beams
        dict(name="beam_one_request", op="beam", B=1, W=4, vocab=32000, take=4, dtype="bf16", mask=False, finished=False),
        # a batch under constraints (a mask of allowed tokens), some hypotheses finished, an odd vocabulary
        dict(name="beam_masked_fp32", op="beam", B=8, W=5, vocab=50021, take=10, dtype="fp32", mask=True, finished=True),
        # many requests over a large vocabulary
        dict(name="beam_large", op="beam", B=64, W=8, vocab=131072, take=8, dtype="bf16", mask=False, finished=True),
        # the states of two layers, and the short convolutions' last inputs beside them, follow the beams
        dict(name="reorder_batch", op="reorder", B=16, W=8, Hv=32, K=128, V=128, layers=2, tail=8192 + 4096),
        # one request's beams, one layer
        dict(name="reorder_one_request", op="reorder", B=1, W=4, Hv=32, K=128, V=128, layers=1, tail=0),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["step", "tree", "beam", "reorder"])
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        Hq = rng.choice([1, 2, 4, 8, 16])
        Hv = Hq * rng.choice([1, 2, 3, 4])
        K, V = rng.choice([(128, 128), (128, 128), (128, 64), (64, 128), (64, 64)])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        if op == "step":
            c = dict(op=op, B=_spread(rng, 1, 160), T=_spread(rng, 1, 8), Hq=Hq, Hv=Hv, K=K, V=V, dtype=dtype,
                     path=rng.random() < 0.3)
        elif op == "tree":
            c = dict(op=op, B=_spread(rng, 1, 96), T=_spread(rng, 1, 64), Hq=Hq, Hv=Hv, K=K, V=V, dtype=dtype)
        elif op == "beam":
            W = _spread(rng, 1, 16)
            c = dict(op=op, B=_spread(rng, 1, 64), W=W, vocab=_spread(rng, 1000, 131072), take=W * rng.choice([1, 2]),
                     dtype=dtype, mask=rng.random() < 0.3, finished=rng.random() < 0.5)
        else:
            c = dict(op=op, B=_spread(rng, 1, 24), W=_spread(rng, 2, 16), Hv=Hv, K=K, V=V, layers=rng.choice([1, 2, 4]),
                     tail=rng.choice([0, 2 * Hq * K + Hv * V, rng.randint(1, 20000)]))
        if work(c)["bytes"] <= most:
            return c


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    op, s = case["op"], dict(case)
    if op in ("step", "tree"):
        B, T, Hq, Hv, K, V = (case[n] for n in ("B", "T", "Hq", "Hv", "K", "V"))
        # q, k and v of a token lie side by side, as one projection writes them; q and k are normalised
        nq = Hq * K
        packed = torch.empty(B, T, 2 * nq + Hv * V, device="cuda", dtype=_dtype(case))
        s["q"] = packed[..., :nq].view(B, T, Hq, K)
        s["k"] = packed[..., nq:2 * nq].view(B, T, Hq, K)
        s["v"] = packed[..., 2 * nq:].view(B, T, Hv, V)
        for name in ("q", "k"):
            x = normal(B, T, Hq, K)
            s[name].copy_(x / x.norm(dim=-1, keepdim=True))
        s["v"].copy_(normal(B, T, Hv, V))
        s["g"] = -torch.nn.functional.softplus(normal(B, T, Hv))
        s["beta"] = torch.sigmoid(normal(B, T, Hv))
        slots = B + B // 4 + 1
        s["state"] = 0.1 * normal(slots, Hv, K, V)
        s["slots"] = torch.randperm(slots, device="cuda", generator=gen)[:B].to(torch.int32)
        if op == "tree":  # a node's parent is an earlier node or, -1, the state
            s["parents"] = ((uniform(B, T) * (torch.arange(T, device="cuda") + 1)).long() - 1).to(torch.int32)
        s["accepted"] = None
        if case.get("path"):  # the nodes that were accepted, in order: at least one; the end is marked by -1
            order = torch.sort(uniform(B, T), dim=1).indices
            count = (uniform(B, 1) * T).long() + 1
            keep = torch.arange(T, device="cuda") < count
            path = torch.sort(torch.where(keep, order, T), dim=1).values
            s["accepted"] = torch.where(path < T, path, -1).to(torch.int32)
    elif op == "beam":
        B, W, N = case["B"], case["W"], case["vocab"]
        s["logits"] = (4 * normal(B, W, N)).to(_dtype(case))
        s["scores"] = -10 * uniform(B, W)
        s["finished"] = uniform(B, W) < 0.15 if case["finished"] else None
        s["mask"] = None
        if case["mask"]:
            s["mask"] = uniform(B, W, N) < 0.4
            s["mask"][B // 2, W // 2] = False  # one hypothesis that may not be continued at all
    else:
        B, W = case["B"], case["W"]
        s["states"] = [0.1 * normal(B * W, case["Hv"], case["K"], case["V"]) for _ in range(case["layers"])]
        if case["tail"]:
            s["states"] += [normal(B * W, 3, case["tail"]).to(torch.bfloat16) for _ in range(case["layers"])]
        s["parents"] = (uniform(B, W) * W).long().clamp(max=W - 1).to(torch.int32)
    return s


# ---- the plain forms ------------------------------------------------------------------------------


def _heads(x, Hv):
    """[B, T, H, D] -> [B, Hv, T, D] in 32 bits, a query / key head for each of its value heads."""
    x = x.float().transpose(1, 2)
    return x if x.shape[1] == Hv else x.repeat_interleave(Hv // x.shape[1], dim=1)


def _sum_powers(M, x, reach):
    """(1 + M + M^2 + ...) x for a strictly lower M of at most `reach` rows."""
    x = x + M @ x
    return x if reach <= 2 else _sum_powers(M @ M, x, (reach + 1) // 2)


def _closure(A, reach):
    """Ancestors at any distance, from the nodes themselves and their parents."""
    return A if reach <= 1 else _closure(((A @ A) > 0).float(), (reach + 1) // 2)


def _block(q, k, v, g, beta, S, above):
    """A block of tokens over a state: (what the state and the block answer, the corrections, the decay from
    each token to each, from the state to each).  above[t, i]: token i is t or comes before it."""
    T = k.shape[2]
    gsum = above @ g.unsqueeze(-1)
    decay = torch.exp(torch.where(above > 0, gsum - gsum.transpose(-1, -2), float("-inf")))
    reach = torch.exp(gsum)
    r = beta.unsqueeze(-1) * (v - reach * (k @ S))
    if T > 1:
        L = torch.tril(beta.unsqueeze(-1) * decay * (k @ k.transpose(-1, -2)), -1)
        r = _sum_powers(-L, r, T)
    o = None
    if q is not None:
        o = reach * (q @ S) + (decay * (q @ k.transpose(-1, -2))) @ r
    return o, r, decay, reach


def _plain_step(s):
    q, k, v, g, beta = s["q"], s["k"], s["v"], s["g"], s["beta"]
    Hv, K = s["Hv"], s["K"]
    if s["accepted"] is not None:
        at = s["accepted"].long().clamp(min=0)
        live = (s["accepted"] >= 0).unsqueeze(-1)
        row = torch.arange(at.shape[0], device=at.device).unsqueeze(1)
        q, k, v, g, beta = None, k[row, at], v[row, at], g[row, at] * live, beta[row, at] * live
    T = k.shape[1]
    slots = s["slots"].long()
    S = s["state"][slots]
    k, v = _heads(k, Hv), v.float().transpose(1, 2)
    above = torch.tril(torch.ones(T, T, device=k.device))
    o, r, decay, reach = _block(None if q is None else _heads(q, Hv), k, v, g.transpose(1, 2), beta.transpose(1, 2),
                                S, above)
    S = reach[:, :, -1:] * S + (k * decay[:, :, -1].unsqueeze(-1)).transpose(-1, -2) @ r
    s["state"][slots] = S
    if o is None:
        return {"state": s["state"]}
    return {"o": (o * K ** -0.5).transpose(1, 2).to(s["q"].dtype), "state": s["state"]}


def _plain_tree(s):
    Hv, K, T = s["Hv"], s["K"], s["T"]
    node = torch.arange(T, device="cuda")
    parent = s["parents"].long().unsqueeze(-1)
    above = _closure(((parent == node) | (node.unsqueeze(-1) == node)).float(), T).unsqueeze(1)
    o, _, _, _ = _block(_heads(s["q"], Hv), _heads(s["k"], Hv), s["v"].float().transpose(1, 2), s["g"].transpose(1, 2),
                        s["beta"].transpose(1, 2), s["state"][s["slots"].long()], above)
    return {"o": (o * K ** -0.5).transpose(1, 2).to(s["q"].dtype)}


def _plain_beam(s):
    B, W, N, take = s["B"], s["W"], s["vocab"], s["take"]
    x = s["logits"].float()
    if s["mask"] is not None:
        x = torch.where(s["mask"], x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    norm = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    cand = s["scores"].unsqueeze(-1) + (x - norm)
    if s["finished"] is not None:
        cand[s["finished"]] = float("-inf")
        cand[..., 0] = torch.where(s["finished"], s["scores"], cand[..., 0])
    cand = torch.where(torch.isnan(cand), float("-inf"), cand) + 0.0
    # one whole number orders by value, then by the lower index
    bits = cand.view(B, W * N).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32
    order += 0xFFFFFFFF - torch.arange(W * N, device=x.device)
    flat = 0xFFFFFFFF - (torch.topk(order, take, dim=-1).values & 0xFFFFFFFF)
    score = cand.view(B, W * N).gather(1, flat)
    return _answer(s, score, flat)


def _answer(s, score, flat):
    """Scores, tokens and parents of the chosen candidates; where nothing is left to choose, the token is -1 and
    the parent the place itself."""
    parent = flat // s["vocab"]
    token = flat % s["vocab"]
    if s["finished"] is not None:
        token = torch.where(s["finished"].gather(1, parent), _SETTLED, token)
    none = score == float("-inf")
    place = torch.arange(s["take"], device=score.device) % s["W"]
    return {"scores": score, "tokens": torch.where(none, _SETTLED, token).to(torch.int32),
            "parents": torch.where(none, place, parent).to(torch.int32)}


def _plain_reorder(s):
    B, W = s["B"], s["W"]
    source = (s["parents"].long() + W * torch.arange(B, device="cuda").unsqueeze(1)).view(-1)
    return [x.copy_(x[source]) for x in s["states"]]


# ---- one pass -------------------------------------------------------------------------------------


def run(state):
    s = state
    if not own:
        return {"step": _plain_step, "tree": _plain_tree, "beam": _plain_beam, "reorder": _plain_reorder}[s["op"]](s)
    import gated_delta_rule_50_gb300 as gdn
    if s["op"] == "step":
        if s["accepted"] is not None:
            gdn.recurrent_gated_delta_rule(None, s["k"], s["v"], s["g"], s["beta"], s["state"], state_indices=s["slots"],
                                           token_indices=s["accepted"])
            return {"state": s["state"]}
        o = gdn.recurrent_gated_delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"],
                                           state_indices=s["slots"])
        return {"o": o, "state": s["state"]}
    if s["op"] == "tree":
        return {"o": gdn.tree_gated_delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], s["parents"], s["state"],
                                               state_indices=s["slots"])}
    if s["op"] == "beam":
        scores, tokens, parents = gdn.beam_search_step(s["logits"], s["scores"], finished=s["finished"], mask=s["mask"],
                                                       num_candidates=s["take"])
        return {"scores": scores, "tokens": tokens, "parents": parents}
    gdn.reorder_states(s["states"], s["parents"])
    return s["states"]


def work(case):
    op = case["op"]
    if op in ("step", "tree"):
        B, T, Hq, Hv, K, V = (case[n] for n in ("B", "T", "Hq", "Hv", "K", "V"))
        size = 2 if case["dtype"] == "bf16" else 4
        state = B * Hv * K * V * 4
        if op == "tree":
            tokens = B * T
            io = tokens * ((2 * Hq * K + 2 * Hv * V) * size + 8 * Hv + 4)
            # q and k against the state; every pair of a node and one above it, about half of the square at most
            return {"bytes": state + io, "flops": tokens * (Hv * (4 * K * V + 2 * T * V) + Hq * 2 * T * K)}
        if case["path"]:  # lengths are spread evenly over 1 .. T
            tokens = B * (T + 1) / 2
            return {"bytes": 2 * state + tokens * ((Hq * K + Hv * V) * size + 8 * Hv + 4), "flops": tokens * Hv * 5 * K * V}
        tokens = B * T
        return {"bytes": 2 * state + tokens * ((2 * Hq * K + 2 * Hv * V) * size + 8 * Hv), "flops": tokens * Hv * 7 * K * V}
    if op == "beam":
        rows = case["B"] * case["W"] * (0.85 if case["finished"] else 1)
        each = (2 if case["dtype"] == "bf16" else 4) + (1 if case["mask"] else 0)
        return {"bytes": rows * case["vocab"] * each + case["B"] * (case["W"] * 5 + case["take"] * 12),
                "flops": rows * case["vocab"] * 4}
    B, W = case["B"], case["W"]
    slot = case["layers"] * (case["Hv"] * case["K"] * case["V"] * 4 + 3 * case["tail"] * 2)
    # parents are uniform: a slot is written where its parent is another, and read where another follows it
    written, read = 1 - 1 / W, 1 - (1 - 1 / W) ** (W - 1)
    return {"bytes": B * W * slot * (written + read), "flops": 0}


# ---- the definitions in 64 bits --------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op, B, f64 = case["op"], case["B"], torch.float64

    def advance(S, k, v, g, beta):
        """One token, each head: S <- e^g S + k (beta (v - e^g S^T k))^T.  S [H, K, V], k [H, K], v [H, V]."""
        S = S * torch.exp(g)[:, None, None]
        miss = v - (S * k.unsqueeze(-1)).sum(-2)
        return S + k.unsqueeze(-1) * (beta.unsqueeze(-1) * miss).unsqueeze(-2)

    def answer(S, q):
        return (S * q.unsqueeze(-1)).sum(-2) * case["K"] ** -0.5

    if op in ("step", "tree"):
        G = case["Hv"] // case["Hq"]
        o = torch.zeros(B, case["T"], case["Hv"], case["V"], dtype=f64, device="cuda")
        state = s["state"].double()
        slots = s["slots"].tolist()
        for b in range(B):
            q, k = (s[n][b].double().repeat_interleave(G, 1) for n in ("q", "k"))
            v, g, beta = (s[n][b].double() for n in ("v", "g", "beta"))
            if op == "tree":  # the state, then the state after each node
                reached = [state[slots[b]]]
                for t, parent in enumerate(s["parents"][b].tolist()):
                    reached.append(advance(reached[parent + 1], k[t], v[t], g[t], beta[t]))
                    o[b, t] = answer(reached[-1], q[t])
                continue
            S = state[slots[b]]
            for t in range(case["T"]) if s["accepted"] is None else [t for t in s["accepted"][b].tolist() if t >= 0]:
                S = advance(S, k[t], v[t], g[t], beta[t])
                o[b, t] = answer(S, q[t])
            state[slots[b]] = S
        return {"o": o} if op == "tree" else {"state": state} if case["path"] else {"o": o, "state": state}
    if op == "beam":
        x = s["logits"].double()
        if s["mask"] is not None:
            x = x.masked_fill(~s["mask"], float("-inf"))
        cand = torch.log_softmax(x, -1) + s["scores"].double().unsqueeze(-1)
        cand = cand.masked_fill(cand.isnan(), float("-inf"))
        if s["finished"] is not None:
            cand = cand.masked_fill(s["finished"].unsqueeze(-1), float("-inf"))
            cand[..., 0] = torch.where(s["finished"], s["scores"].double(), cand[..., 0])
        score, flat = torch.sort(cand.flatten(1), dim=1, descending=True, stable=True)
        score, flat = score[:, :case["take"]], flat[:, :case["take"]]
        parents, tokens = flat // case["vocab"], flat % case["vocab"]
        for b in range(B):
            for j in range(case["take"]):
                w = int(parents[b, j])
                if score[b, j] == float("-inf"):
                    tokens[b, j], parents[b, j] = _SETTLED, j % case["W"]
                elif s["finished"] is not None and s["finished"][b, w]:
                    tokens[b, j] = _SETTLED
        return {"scores": score.contiguous(), "tokens": tokens, "parents": parents}
    W, parents, out = case["W"], s["parents"].tolist(), []
    for x in s["states"]:
        y = x.double()
        for b in range(B):
            for i in range(W):
                y[b * W + i] = x[b * W + parents[b][i]].double()
        out.append(y)
    return out

"""Linear attention with a decay for each head, and the sampling of tokens, at sizes of real use.

Each operator is here as plain torch operations (``own`` false) and as the calls a user makes of this
package (``own`` true), on the same inputs:

* ``prompt``: linear attention over whole sequences, padded to one length or packed one after the other
  (``chunk_linear_attention``);
* ``train``: the same with the gradients of q, k, v and the initial state;
* ``step``: new tokens move the sequences' states, held in a pool of slots (``recurrent_linear_attention``);
* ``sample``: one token for each row of logits, by temperature, top-k, top-p and min-p, from a given
  random number (``sample_tokens``).

``own`` is set from outside.
"""
import math

import torch

own = False

_BLOCK = 64  # tokens that the plain form takes at a time


def listed():
    return [
        # a short question of one user: little work, latency counts; an odd number of tokens
        dict(name="prompt_short", op="prompt", B=1, T=97, Hq=32, Hv=32, K=128, V=128, dtype="bf16", packed=False, h0=False),
        # prompts of a serving batch, from which decoding goes on
        dict(name="prompt_batch", op="prompt", B=4, T=4096, Hq=16, Hv=32, K=128, V=128, dtype="bf16", packed=False, h0=False),
        # one long document on few heads, a later part of it: it begins from the state of the part before
        dict(name="prompt_long", op="prompt", B=1, T=32768, Hq=8, Hv=8, K=128, V=128, dtype="bf16", packed=False, h0=True),
        # prompts of very different lengths packed one after the other, one of them empty, one of a single token
        dict(name="prompt_packed", op="prompt", B=13, T=10007, Hq=16, Hv=32, K=128, V=128, dtype="bf16", packed=True, h0=True),
        # 32-bit activations with narrow heads
        dict(name="prompt_fp32_narrow", op="prompt", B=2, T=1000, Hq=4, Hv=8, K=64, V=64, dtype="fp32", packed=False, h0=True),
        # one training step of a small layer with heads of two widths
        dict(name="train_small", op="train", B=1, T=777, Hq=8, Hv=8, K=64, V=128, dtype="bf16", packed=False, h0=True),
        # one training step of a large layer, four value heads to a query head
        dict(name="train_large", op="train", B=2, T=8192, Hq=16, Hv=64, K=128, V=128, dtype="bf16", packed=False, h0=False),
        # one sequence decoding one token: all that counts is latency
        dict(name="step_one_token", op="step", B=1, T=1, Hq=32, Hv=32, K=128, V=128, dtype="bf16"),
        # a serving batch, one token each
        dict(name="step_batch", op="step", B=64, T=1, Hq=16, Hv=32, K=128, V=128, dtype="bf16"),
        # one request: a vocabulary of ordinary size, the usual filters
        dict(name="sample_one", op="sample", B=1, vocab=32000, dtype="bf16", mask=False, top_k=True, top_p=True, min_p=False),
        # a batch under constraints (a mask of allowed tokens), an odd vocabulary
        dict(name="sample_masked_fp32", op="sample", B=8, vocab=50021, dtype="fp32", mask=True, top_k=False, top_p=True, min_p=True),
        # many requests over a large vocabulary, every filter
        dict(name="sample_large", op="sample", B=64, vocab=131072, dtype="bf16", mask=False, top_k=True, top_p=True, min_p=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "step", "sample"])
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        Hq = rng.choice([1, 2, 4, 8, 16, 32])
        Hv = Hq * rng.choice([1, 1, 2, 3, 4])
        K, V = rng.choice([(128, 128), (128, 128), (128, 64), (64, 128), (64, 64)])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        c = dict(op=op, B=_spread(rng, 1, 16), T=_spread(rng, 1, 16384), Hq=Hq, Hv=Hv, K=K, V=V, dtype=dtype,
                 packed=rng.random() < 0.4, h0=rng.random() < 0.5)
        if c["packed"]:  # T counts the tokens of all sequences
            c["T"] = max(c["T"], c["B"])
        if op == "step":
            c = dict(op=op, B=_spread(rng, 1, 160), T=_spread(rng, 1, 8), Hq=Hq, Hv=Hv, K=K, V=V, dtype=dtype)
        elif op == "sample":
            c = dict(op=op, B=_spread(rng, 1, 256), vocab=_spread(rng, 1000, 200000), dtype=dtype,
                     mask=rng.random() < 0.3, top_k=rng.random() < 0.6, top_p=rng.random() < 0.6, min_p=rng.random() < 0.4)
        # 32-bit activations come at moderate sizes
        limit = most / 4 if dtype == "fp32" and op in ("prompt", "train") else most
        if work(c)["bytes"] <= limit:
            return c


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    """The lengths of the sequences: all T, or, packed, of very different sizes that sum to T."""
    B, T = case["B"], case["T"]
    if not case["packed"]:
        return [T] * B
    share = [1.7 ** (i * 5 % B) if i * 5 % B < 9 else 0.0 for i in range(B)]
    got = [int(T * x / sum(share)) for x in share]
    if B > 2:
        got[1] = min(T, 1)
    got[-1] += T - sum(got)
    return got


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    op, B, s = case["op"], case["B"], dict(case)
    if op == "sample":
        N = case["vocab"]
        s["logits"] = (3 * normal(B, N)).to(_dtype(case))
        s["random"] = uniform(B)
        s["temperature"] = 0.5 + uniform(B)
        s["temperature"][B // 2 :][::7][1:] = 0.0  # some requests in a batch are greedy
        s["top_k"] = (1 + 100 * uniform(B)).to(torch.int32) if case["top_k"] else None
        s["top_p"] = 0.7 + 0.3 * uniform(B) if case["top_p"] else None
        s["min_p"] = 0.1 * uniform(B) if case["min_p"] else None
        s["mask"] = None
        if case["mask"]:
            s["mask"] = uniform(B, N) < 0.4
            if B > 1:
                s["mask"][B // 2] = False  # one request for which nothing is allowed
        return s
    T, Hq, Hv, K, V = (case[n] for n in ("T", "Hq", "Hv", "K", "V"))
    rows = 1 if case.get("packed") else B
    # the slopes of such layers: from heads that forget within a few tokens to heads that hardly do
    s["g"] = -torch.exp2(-8 * (torch.arange(Hv, device="cuda") + uniform(1)) / Hv).float()
    if op == "train":
        s["q"], s["k"] = (normal(rows, T, Hq, K).to(_dtype(case)) for _ in range(2))
        s["v"], s["do"] = (normal(rows, T, Hv, V).to(_dtype(case)) for _ in range(2))
    else:  # q, k and v of a token lie side by side, as one projection writes them
        nq = Hq * K
        side = torch.empty(rows, T, 2 * nq + Hv * V, device="cuda", dtype=_dtype(case))
        s["q"] = side[..., :nq].view(rows, T, Hq, K)
        s["k"] = side[..., nq : 2 * nq].view(rows, T, Hq, K)
        s["v"] = side[..., 2 * nq :].view(rows, T, Hv, V)
        s["q"].copy_(normal(rows, T, Hq, K))
        s["k"].copy_(normal(rows, T, Hq, K))
        s["v"].copy_(normal(rows, T, Hv, V))
    if op == "step":
        slots = B + B // 4 + 1
        s["state"] = normal(slots, Hv, K, V)
        s["slots"] = torch.randperm(slots, device="cuda", generator=gen)[:B].to(torch.int32)
        return s
    s["cu"] = None
    if case["packed"]:
        ends = [0]
        for n in _lengths(case):
            ends.append(ends[-1] + n)
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    s["state"] = normal(B, Hv, K, V) if case["h0"] else None
    if op == "train":
        s["dstate"] = normal(B, Hv, K, V) if case["h0"] else None
        s["leaves"] = [s[n].requires_grad_() for n in ("q", "k", "v", "state") if s[n] is not None]
    return s


# ---- the plain forms ------------------------------------------------------------------------------


def _places(s, reverse):
    """Each sequence's tokens, filled up in front to one length of whole blocks: where each place's token lies among
    all tokens [B, L], the token's number within its sequence (negative: there is none), the sequences' lengths."""
    B, T, dev = s["B"], s["T"], s["q"].device
    if s["cu"] is None:
        start = T * torch.arange(B, device=dev)
        length = torch.full((B,), T, device=dev)
        longest = T
    else:
        start, length = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
        longest = max(_lengths(s))
    L = max(1, -(-longest // _BLOCK)) * _BLOCK
    number = torch.arange(L, device=dev) - L + length[:, None]
    at = start[:, None] + (length[:, None] - 1 - number if reverse else number)
    return torch.where(number >= 0, at, 0), number, length


def _attend(s, a, b, c, g, carry, e, reverse=False):
    """sum over i up to r of l^(r - i) (a_r . b_i) c_i + l^(r + e) a_r carry with l = e^g, for each sequence and head, and
    the sum over all its tokens of l^(length - 1 - i) b_i c_i^T + l^length carry; `reverse` counts from the other end."""
    at, number, length = _places(s, reverse)
    there = (number >= 0)[:, None, :, None]
    Hv = g.shape[0]

    def blocks(x):  # [rows, T, H, D] -> [B, Hv, blocks, 64, D] in 32 bits
        x = x.flatten(0, 1)[at].float().transpose(1, 2) * there
        x = x if x.shape[1] == Hv else x.repeat_interleave(Hv // x.shape[1], dim=1)
        return x.unflatten(2, (-1, _BLOCK))

    a, b, c = blocks(a), blocks(b), blocks(c)
    n = a.shape[2]
    g64 = g.double()
    r = torch.arange(_BLOCK, device=g.device)
    between = (g64[:, None, None] * (r[:, None] - r)).masked_fill(r[:, None] < r, float("-inf")).exp().float()
    out = (a @ b.transpose(-1, -2) * between[:, None]) @ c
    # what each block adds to the state by its own end, then what stands before each block
    left = torch.exp(g64[:, None] * (_BLOCK - 1 - r)).float()
    add = (b * left[:, None, :, None]).transpose(-1, -2) @ c
    m = torch.arange(n + 1, device=g.device)
    across = (g64[:, None, None] * _BLOCK * (m[:, None] - 1 - m[:-1])).masked_fill(m[:, None] <= m[:-1], float("-inf")).exp().float()
    before = (across @ add.flatten(-2)).unflatten(-1, add.shape[-2:])
    into = torch.exp(g64[:, None] * (r + 1)).float()
    out = out + into[:, None, :, None] * (a @ before[:, :, :n])
    end = before[:, :, n]
    if carry is not None:
        far = torch.exp(g64[:, None] * (number[:, None].double() + e)).float().unflatten(-1, (-1, _BLOCK))
        out = out + far.unsqueeze(-1) * (a @ carry.unsqueeze(2))
        end = end + torch.exp(g64 * length[:, None].double()).float()[..., None, None] * carry
    return (out.flatten(2, 3), at, number >= 0), end


def _tokens(s, found, heads, D, dtype):
    """Back to [rows, T, heads, D]; heads that share an input sum into it."""
    out, at, there = found
    out = out.transpose(1, 2)
    if out.shape[2] != heads:
        out = out.unflatten(2, (heads, -1)).sum(3)
    y = torch.zeros(s["q"].shape[0] * s["T"], heads, D, device=out.device)
    y[at[there]] = out[there]
    return y.view(s["q"].shape[0], s["T"], heads, D).to(dtype)


def _plain_prompt(s):
    scale = s["K"] ** -0.5
    (o, at, there), end = _attend(s, s["q"], s["k"], s["v"], s["g"], s["state"], 1)
    return {"o": _tokens(s, (o * scale, at, there), s["Hv"], s["V"], s["q"].dtype), "state": end}


@torch.no_grad()
def _plain_train(s):
    K, V, Hq, Hv, g, dtype = s["K"], s["V"], s["Hq"], s["Hv"], s["g"], s["q"].dtype
    scale = K ** -0.5
    q, k, v, do, h0, dht = (s[n] for n in ("q", "k", "v", "do", "state", "dstate"))
    got = _plain_prompt(s)

    def times(found):
        return (found[0] * scale,) + found[1:]

    turn = (lambda x: None if x is None else x.transpose(-1, -2))
    dq, _ = _attend(s, do, v, k, g, turn(h0), 1)
    # the state's gradient enters as it is, the tokens' with the scale
    behind = None if dht is None else dht / scale
    dk, _ = _attend(s, v, do, q, g, turn(behind), 0, reverse=True)
    dv, dh = _attend(s, k, q, do, g, None if dht is None else behind, 0, reverse=True)
    got["dq"] = _tokens(s, times(dq), Hq, K, dtype)
    got["dk"] = _tokens(s, times(dk), Hq, K, dtype)
    got["dv"] = _tokens(s, times(dv), Hv, V, dtype)
    if h0 is not None:  # what a token adds has one more decay on its way to the state before the first
        length = _places(s, True)[2]
        far = torch.exp(g.double() * length[:, None].double()).float()[..., None, None] * dht
        got["dstate"] = torch.exp(g)[:, None, None] * (dh * scale - far) + far
    return got


def _plain_step(s):
    Hv, K, T = s["Hv"], s["K"], s["T"]
    slots = s["slots"].long()
    g = s["g"].double()
    q, k, v = (s[n].float().transpose(1, 2) for n in ("q", "k", "v"))
    if q.shape[1] != Hv:
        q, k = (x.repeat_interleave(Hv // x.shape[1], dim=1) for x in (q, k))
    S = s["state"][slots]
    r = torch.arange(T, device=g.device)
    between = (g[:, None, None] * (r[:, None] - r)).masked_fill(r[:, None] < r, float("-inf")).exp().float()
    into = torch.exp(g[:, None] * (r + 1)).float().unsqueeze(-1)
    o = (q @ k.transpose(-1, -2) * between) @ v + into * (q @ S)
    left = torch.exp(g[:, None] * (T - 1 - r)).float().unsqueeze(-1)
    s["state"][slots] = torch.exp(g * T).float()[:, None, None] * S + (k * left).transpose(-1, -2) @ v
    return {"o": (o * K ** -0.5).transpose(1, 2).to(s["q"].dtype), "state": s["state"]}


def _plain_sample(s):
    x = s["logits"].double()
    N = s["vocab"]
    if s["mask"] is not None:
        x = torch.where(s["mask"], x, float("-inf"))
    greedy = (s["temperature"] == 0).unsqueeze(1)
    heat = torch.where(greedy, 1.0, s["temperature"].unsqueeze(1).double())
    x, order = torch.sort(x, dim=1, descending=True, stable=True)  # equal ones: the lower token first
    top = x[:, :1]
    none = ~(top > float("-inf"))
    mass = torch.exp((x - torch.where(none, 0.0, top)) / heat)
    place = torch.arange(N, device=x.device)
    if s["top_k"] is not None:
        mass = mass * (place < s["top_k"].unsqueeze(1))
    if s["top_p"] is not None:  # the fewest that reach the share
        before = torch.cumsum(mass, 1) - mass
        mass = mass * (before < s["top_p"].unsqueeze(1).double() * mass.sum(1, keepdim=True))
    if s["min_p"] is not None:
        mass = mass * (mass >= s["min_p"].unsqueeze(1).double())
    mass = torch.where(greedy, (place == 0).double(), mass)
    mass = torch.zeros_like(mass).scatter_(1, order, mass)  # by the tokens' numbers
    total = mass.sum(1, keepdim=True)
    token = (torch.cumsum(mass, 1) <= s["random"].unsqueeze(1).double() * total).sum(1, keepdim=True).clamp(max=N - 1)
    share = torch.log(mass.gather(1, token)) - torch.log(total)
    return {"tokens": torch.where(none, -1, token).squeeze(1).to(torch.int32),
            "logprobs": torch.where(none, float("-inf"), share).squeeze(1).float()}


# ---- one pass -------------------------------------------------------------------------------------


def run(state):
    s = state
    if not own:
        return {"prompt": _plain_prompt, "train": _plain_train, "step": _plain_step, "sample": _plain_sample}[s["op"]](s)
    import gated_delta_rule_50_gb300 as gdn
    if s["op"] == "prompt":
        o, end = gdn.chunk_linear_attention(s["q"], s["k"], s["v"], s["g"], initial_state=s["state"],
                                            output_final_state=True, cu_seqlens=s["cu"])
        return {"o": o, "state": end}
    if s["op"] == "train":
        o, end = gdn.chunk_linear_attention(s["q"], s["k"], s["v"], s["g"], initial_state=s["state"],
                                            output_final_state=True, cu_seqlens=s["cu"])
        if s["state"] is None:
            grads = torch.autograd.grad([o], s["leaves"], [s["do"]])
        else:
            grads = torch.autograd.grad([o, end], s["leaves"], [s["do"], s["dstate"]])
        return {"o": o, "state": end, **dict(zip(("dq", "dk", "dv", "dstate"), grads))}
    if s["op"] == "step":
        o = gdn.recurrent_linear_attention(s["q"], s["k"], s["v"], s["g"], s["state"], state_indices=s["slots"])
        return {"o": o, "state": s["state"]}
    tokens, logprobs = gdn.sample_tokens(s["logits"], s["random"], temperature=s["temperature"], top_k=s["top_k"],
                                         top_p=s["top_p"], min_p=s["min_p"], mask=s["mask"])
    return {"tokens": tokens, "logprobs": logprobs}


def work(case):
    op, B = case["op"], case["B"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "sample":
        each = size + (1 if case["mask"] else 0)
        # an exponential, a product and two sums for each logit
        return {"bytes": B * case["vocab"] * each + B * 28, "flops": B * case["vocab"] * 4}
    T, Hq, Hv, K, V = (case[n] for n in ("T", "Hq", "Hv", "K", "V"))
    if op == "step":
        tokens = B * T
        return {"bytes": 2 * B * Hv * K * V * 4 + tokens * (2 * Hq * K + 2 * Hv * V) * size + 4 * Hv,
                "flops": tokens * Hv * 5 * K * V}
    tokens = T if case["packed"] else B * T
    state = B * Hv * K * V * 4
    qk, vo = tokens * Hq * K * size, tokens * Hv * V * size
    # a token's product with the state, its addition to it, and half a block of pairs
    flops = tokens * Hv * (4 * K * V + _BLOCK * (K + V))
    forward = {"bytes": 2 * qk + 2 * vo + state * (2 if case["h0"] else 1), "flops": flops}
    if op == "prompt":
        return forward
    # back: q, k, v and the outputs' gradient in, three gradients out; two states to run through and three products
    back = 4 * qk + 3 * vo + (3 * state if case["h0"] else 0)
    return {"bytes": forward["bytes"] + back, "flops": flops + tokens * Hv * (10 * K * V + _BLOCK * (2 * K + 3 * V))}


# ---- the definitions in 64 bits --------------------------------------------------------------------


def exact(case, seed):
    with torch.no_grad():
        return _exact(case, prepare(case, seed))


def _exact(case, s):
    op, B, f64 = case["op"], case["B"], torch.float64
    if op == "sample":
        tokens, logprobs = [], []
        for b in range(B):
            x = s["logits"][b].double()
            if s["mask"] is not None:
                x[~s["mask"][b]] = float("-inf")
            heat = float(s["temperature"][b])
            if float(x.max()) == float("-inf"):
                tokens.append(-1), logprobs.append(float("-inf"))
                continue
            if heat == 0:
                tokens.append(int((x == x.max()).nonzero()[0])), logprobs.append(0.0)
                continue
            best = torch.argsort(-x, stable=True)  # equal ones keep their order
            if s["top_k"] is not None:
                best = best[: int(s["top_k"][b])]
            p = torch.softmax(x[best] / heat, 0)
            if s["top_p"] is not None:
                share, count = 0.0, 0
                sums = torch.cumsum(p, 0).tolist()
                while count < len(sums) and share < float(s["top_p"][b]):
                    share, count = sums[count], count + 1
                best, p = best[:count], p[:count]
            if s["min_p"] is not None:
                best = best[p >= float(s["min_p"][b]) * p[0]]
            best = torch.sort(best).values
            y = x[best] / heat
            p = torch.softmax(y, 0)
            at = int((torch.cumsum(p, 0) <= float(s["random"][b])).sum())
            at = min(at, len(best) - 1)
            others = torch.cat([y[:at], y[at + 1:]])
            # log of a share near 1 by what is left of it
            rest = float(torch.exp(others - y[at]).sum()) if len(others) else 0.0
            tokens.append(int(best[at])), logprobs.append(-math.log1p(rest))
        return {"tokens": torch.tensor(tokens), "logprobs": torch.tensor(logprobs, dtype=f64)}
    T, Hq, Hv, K, V = (case[n] for n in ("T", "Hq", "Hv", "K", "V"))
    G, scale = Hv // Hq, K ** -0.5
    decay = torch.exp(s["g"].double())[:, None, None]
    rows = s["q"].shape[0]

    def heads(x):
        return x.double().repeat_interleave(G, 2) if x.shape[2] != Hv else x.double()

    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])
    if op == "step":
        S = s["state"].double()
        at = s["slots"].long()
        now, o = S[at], torch.zeros(B, T, Hv, V, dtype=f64, device="cuda")
        for t in range(T):
            now = decay * now + k[:, t, :, :, None] * v[:, t, :, None, :]
            o[:, t] = scale * (now * q[:, t, :, :, None]).sum(-2)
        S[at] = now
        return {"o": o, "state": S}
    o = torch.zeros(rows, T, Hv, V, dtype=f64, device="cuda")
    zero = torch.zeros(B, Hv, K, V, dtype=f64, device="cuda")
    h0 = zero if s["state"] is None else s["state"].double()
    # sequences of one length go side by side, packed ones one after the other
    spans, first = [], 0
    for b, n in enumerate(_lengths(case) if case["packed"] else [T]):
        spans.append((slice(b, b + 1) if case["packed"] else slice(None), first, first + n))
        first += n
    end = zero.clone()
    if op == "train":
        do = s["do"].double()
        dht = zero if s["dstate"] is None else s["dstate"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dh0 = zero.clone()
    for which, lo, hi in spans:
        S = h0[which].clone()
        for t in range(lo, hi):
            S.mul_(decay).addcmul_(k[:, t, :, :, None], v[:, t, :, None, :])
            o[:, t] = scale * torch.einsum("bhkv,bhk->bhv", S, q[:, t])
            if op == "train":
                dq[:, t] = scale * torch.einsum("bhkv,bhv->bhk", S, do[:, t])
        end[which] = S
        if op == "train":
            D = dht[which].clone()
            for t in range(hi - 1, lo - 1, -1):
                D.addcmul_(q[:, t, :, :, None], do[:, t, :, None, :], value=scale)
                dk[:, t] = torch.einsum("bhkv,bhv->bhk", D, v[:, t])
                dv[:, t] = torch.einsum("bhkv,bhk->bhv", D, k[:, t])
                D.mul_(decay)
            dh0[which] = D
    got = {"o": o, "state": end}
    if op == "train":
        got["dq"], got["dk"] = (x.unflatten(2, (Hq, G)).sum(3) for x in (dq, dk))
        got["dv"] = dv
        if s["state"] is not None:
            got["dstate"] = dh0
    return got

"""Linear attention with a decay for each head against the recurrence in 64 bits: forward, backward, token by token.

Tolerances are those of ``parity.py``: fp32 1e-5 * RMS; bf16 outputs 2e-3 * RMS before their rounding.  The fp32 states
of bf16 inputs are held to 1e-5 * RMS too: their operands are split into parts that keep 24 bits, and an element sums at
most a few thousand products whose errors of 2^-23 each are independent."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from parity import BF16_TOL, FP32_TOL, check

pytestmark = pytest.mark.gpu
bf16, f32, f64 = torch.bfloat16, torch.float32, torch.float64


def make(B, T, Hq, Hv, K, V, dtype, seed=0, h0=True, packed=False):
    """Inputs on the GPU; packed: q, k and v of a token side by side."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    nq = Hq * K
    if packed:
        side = normal(B, T, 2 * nq + Hv * V).to(dtype).cuda()
        q, k = side[..., :nq].view(B, T, Hq, K), side[..., nq:2 * nq].view(B, T, Hq, K)
        v = side[..., 2 * nq:].view(B, T, Hv, V)
    else:
        q, k, v = (normal(B, T, *s).to(dtype).cuda() for s in ((Hq, K), (Hq, K), (Hv, V)))
    g = -torch.exp2(-8 * torch.rand(Hv, generator=gen))
    g[0] = 0.0
    x = dict(q=q, k=k, v=v, g=g.cuda(), scale=K ** -0.5, h0=None, dht=None)
    x["do"] = normal(B, T, Hv, V).to(dtype).cuda()
    if h0:
        x["h0"], x["dht"] = normal(B, Hv, K, V).cuda(), normal(B, Hv, K, V).cuda()
    return x


def reference(x, spans=None, backward=False):
    """The recurrence token by token in 64 bits; spans: [(row, first, last + 1)] for each state (default: whole rows)."""
    q, k, v, do = (x[n].to(f64) for n in ("q", "k", "v", "do"))
    G = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(G, 2), k.repeat_interleave(G, 2)
    B, T, Hv, V = v.shape
    K = q.shape[3]
    spans = spans or [(b, 0, T) for b in range(B)]
    decay = torch.exp(torch.zeros(Hv, device="cuda") if x["g"] is None else x["g"]).to(f64)[:, None, None]
    if x["g"] is not None:
        decay = torch.exp(x["g"].to(f64))[:, None, None]
    zero = torch.zeros(len(spans), Hv, K, V, dtype=f64, device="cuda")
    h0 = zero if x["h0"] is None else x["h0"].to(f64)
    dht = zero if x["dht"] is None else x["dht"].to(f64)
    o, ht, dq, dk, dv, dh0 = torch.zeros_like(v), zero.clone(), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), zero.clone()
    for n, (b, lo, hi) in enumerate(spans):
        S = h0[n].clone()
        for t in range(lo, hi):
            S = decay * S + k[b, t, :, :, None] * v[b, t, :, None, :]
            o[b, t] = x["scale"] * (S * q[b, t, :, :, None]).sum(-2)
            if backward:
                dq[b, t] = x["scale"] * (S * do[b, t, :, None, :]).sum(-1)
        ht[n] = S
        if backward:
            D = dht[n].clone()
            for t in reversed(range(lo, hi)):
                D = D + x["scale"] * q[b, t, :, :, None] * do[b, t, :, None, :]
                dk[b, t] = (D * v[b, t, :, None, :]).sum(-1)
                dv[b, t] = (D * k[b, t, :, :, None]).sum(-2)
                D = decay * D
            dh0[n] = D
    Hq = Hv // G
    return dict(o=o, ht=ht, dq=dq.unflatten(2, (Hq, G)).sum(3), dk=dk.unflatten(2, (Hq, G)).sum(3), dv=dv, dh0=dh0)


def verify(name, got, ref, io):
    assert got.dtype == (f32 if name in ("ht", "dh0") else io)
    check(name, got, ref, io, got.dtype, tol=FP32_TOL if got.dtype == f32 else BF16_TOL)


CASES = [  # B, T, Hq, Hv, K, V, dtype
    (1, 1, 1, 1, 64, 64, f32), (2, 65, 2, 4, 128, 128, f32), (1, 300, 1, 3, 64, 128, f32), (2, 33, 2, 2, 128, 64, f32),
    (1, 1, 1, 1, 128, 128, bf16), (2, 64, 2, 4, 128, 128, bf16), (3, 63, 1, 2, 128, 128, bf16), (1, 129, 2, 6, 128, 128, bf16),
    (2, 200, 2, 2, 64, 64, bf16), (1, 777, 2, 4, 64, 128, bf16), (2, 130, 1, 4, 128, 64, bf16), (40, 70, 2, 8, 128, 128, bf16),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, packed):
    x = make(*case, seed=sum(case[:6]), packed=packed)
    o, ht = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], output_final_state=True)
    ref = reference(x)
    verify("o", o, ref["o"], case[6])
    verify("ht", ht, ref["ht"], case[6])


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    x = make(*case, seed=1 + sum(case[:6]))
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], output_final_state=True)
    grads = torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]])
    with torch.no_grad():
        ref = reference(x, backward=True)
    for name, got in zip(("dq", "dk", "dv", "dh0"), grads):
        verify(name, got, ref[name], case[6])


@pytest.mark.parametrize("G", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("K", [64, 128])
def test_shared_heads(G, K):
    """Gradients of q and k are sums over the value heads that share them, in groups that the kernel sums itself and others."""
    x = make(2, 150, 2, 2 * G, K, 128, bf16, seed=G + K)
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], output_final_state=True)
    grads = torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]])
    with torch.no_grad():
        ref = reference(x, backward=True)
    for name, got in zip(("dq", "dk", "dv", "dh0"), grads):
        verify(name, got, ref[name], bf16)


def packed_case(lengths, Hq, Hv, K, V, dtype, seed, T=None):
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    x = make(1, T or ends[-1], Hq, Hv, K, V, dtype, seed=seed, h0=False)
    gen = torch.Generator().manual_seed(seed + 1)
    x["h0"], x["dht"] = (torch.randn(len(lengths), Hv, K, V, generator=gen).cuda() for _ in range(2))
    return x, torch.tensor(ends, dtype=torch.int32).cuda(), [(0, a, b) for a, b in zip(ends, ends[1:])]


PACKED = [  # lengths, Hq, Hv, K, V, dtype
    ([5, 0, 1, 130, 64], 2, 4, 128, 128, bf16), ([300], 1, 2, 128, 128, bf16), ([64, 65, 63], 2, 2, 64, 128, bf16),
    ([1500, 10, 3, 200, 0, 70, 1], 4, 8, 128, 128, bf16), ([40, 90], 1, 3, 64, 64, f32), ([900, 0, 31, 700, 2], 2, 4, 128, 64, f32),
    ([3, 1] * 30 + [100], 1, 2, 128, 128, bf16), ([2100, 40, 40, 300], 24, 24, 64, 64, bf16),
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: "%d_%s" % (len(c[0]), "_".join(map(str, c[1:]))))
def test_packed(case):
    x, cu, spans = packed_case(*case, seed=len(case[0]))
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = gdn.chunk_linear_attention(x["q"], x["k"], x["v"], x["g"], initial_state=x["h0"], output_final_state=True, cu_seqlens=cu)
    grads = torch.autograd.grad([o, ht], leaves, [x["do"], x["dht"]])
    with torch.no_grad():
        ref = reference(x, spans, backward=True)
    verify("o", o, ref["o"], case[5])
    verify("ht", ht, ref["ht"], case[5])
    for name, got in zip(("dq", "dk", "dv", "dh0"), grads):
        verify(name, got, ref[name], case[5])

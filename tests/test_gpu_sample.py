"""Sampling against the definition in 64 bits: tokens equal, logprobs to fp32's rounding."""
import math

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


def drawn(logits, u, temperature, top_k, top_p, min_p, allowed):
    """(token, logprob) of one row; in 64 bits, on the CPU."""
    x = logits.double()
    x[~allowed] = -math.inf
    if not bool((x > -math.inf).any()):
        return -1, -math.inf
    if temperature == 0:
        return int((x == x.max()).nonzero()[0]), 0.0
    order = torch.argsort(-x, stable=True)
    order = order[x[order] > -math.inf]
    if top_k > 0:
        order = order[:top_k]
    p = torch.softmax(x[order] / temperature, 0)
    if top_p < 1:
        before = torch.cumsum(p, 0) - p
        count = max(1, int((before < top_p).sum()))
        order, p = order[:count], p[:count]
    if min_p > 0:
        order = order[p >= min(min_p, 1.0) * p[0]]
    order = torch.sort(order).values
    y = x[order] / temperature
    p = torch.softmax(y, 0)
    at = min(int((torch.cumsum(p, 0) <= u).sum()), len(order) - 1)
    others = torch.cat([y[:at], y[at + 1:]])
    return int(order[at]), -math.log1p(float(torch.exp(others - y[at]).sum())) if len(others) else 0.0


def verify(got, logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mask=None):
    tokens, logprobs = (t.cpu() for t in got)
    assert tokens.dtype == torch.int32 and logprobs.dtype == f32
    B, N = logits.shape

    def row(v, b):  # as the call takes it: numbers become fp32
        return v[b].item() if isinstance(v, torch.Tensor) else v if isinstance(v, int) else torch.tensor(v, dtype=f32).item()

    allowed = torch.ones(B, N, dtype=torch.bool) if mask is None else mask.cpu().expand(B, N)
    x, u = logits.cpu(), u.cpu()
    for b in range(B):
        token, share = drawn(x[b].float(), u[b].item(), row(temperature, b), row(top_k, b), row(top_p, b), row(min_p, b), allowed[b])
        assert tokens[b] == token, (b, int(tokens[b]), token)
        # the logarithm of a quotient of two fp32 numbers, or a difference of two such: a few roundings of the larger
        got_share = logprobs[b].item()
        assert got_share == share or abs(got_share - share) <= 8 * 2.0 ** -24 * max(abs(share), 1e-30) + (
            0 if share > -0.69 else 2.0 ** -22 * 4), (b, got_share, share)


def inputs(B, N, dtype, seed, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(B, N, generator=gen)).to(dtype).cuda(), torch.rand(B, generator=gen).cuda(), gen


CASES = [dict(), dict(top_k=1), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=3000, top_p=0.8),
         dict(top_k=40, top_p=0.7, min_p=0.02), dict(top_p=0.999, min_p=1e-6), dict(top_k=5000), dict(min_p=2.0), dict(top_p=0.0)]


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("N", [1, 2, 9, 1000, 5001, 50021])
@pytest.mark.parametrize("filters", CASES, ids=str)
def test_filters(filters, N, dtype):
    logits, u, _ = inputs(7, N, dtype, N)
    verify(gdn.sample_tokens(logits, u, temperature=1.3, **filters), logits, u, temperature=1.3, **filters)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("B", [1, 3, 40, 100, 200])
def test_rows_of_their_own(B, dtype):
    N = 20011
    logits, u, gen = inputs(B, N, dtype, B)
    heat = 0.3 + torch.rand(B, generator=gen)
    heat[::5] = 0
    k = torch.randint(-1, 3000, (B,), generator=gen).to(torch.int32)
    p = 0.5 + 0.6 * torch.rand(B, generator=gen)
    m = 0.1 * torch.rand(B, generator=gen) - 0.02
    mask = torch.rand(B, N, generator=gen) < 0.5
    mask[B // 2] = False
    got = gdn.sample_tokens(logits, u, heat.cuda(), k.cuda(), p.cuda(), m.cuda(), mask.cuda())
    verify(got, logits, u, heat, k, p, m, mask)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("filters", [dict(), dict(top_k=3000), dict(top_k=7), dict(top_p=0.37), dict(top_k=4000, top_p=0.61)], ids=str)
def test_equal_logits(filters, dtype):
    """More equal ones than the list holds: cuts among them go by the lower token."""
    N = 20000
    logits, u, gen = inputs(4, N, dtype, 3)
    logits[0] = 1.5
    logits[1] = torch.round(logits[1].float() / 4).to(dtype)
    logits[2, : N // 2] = 2.0
    verify(gdn.sample_tokens(logits, u, **filters), logits, u, **filters)

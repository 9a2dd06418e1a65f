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


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("N,B", [(1 << 20, 2), (300000, 3), (40000, 200)])
def test_large(N, B, dtype):
    """The longest vocabulary (slices that are read again in every pass), and many rows."""
    logits, u, gen = inputs(B, N, dtype, 5, spread=2.0)
    kinds = dict(temperature=1.2, top_k=2000, top_p=0.9, min_p=0.001)
    verify(gdn.sample_tokens(logits, u, **kinds), logits, u, **kinds)
    verify(gdn.sample_tokens(logits, u, top_p=0.95), logits, u, top_p=0.95)


def test_layouts():
    """Rows of a wider tensor, masks for all rows and for all tokens of a row, parameters of other types."""
    wide, u, gen = inputs(6, 7001, bf16, 6)
    logits = wide[:, 3:5004]
    mask = (torch.rand(1, 5001, generator=gen) < 0.5).cuda()
    u2 = torch.stack([u, u], 1)[:, 0]
    heat = torch.full((6,), 0.75, dtype=torch.float64).cuda()
    k = torch.tensor([1, 5, 2 ** 40, -3, 100, 0]).cuda()
    got = gdn.sample_tokens(logits, u2, heat, k, 0.875, None, mask)
    verify(got, logits, u, 0.75, k.clamp(max=10 ** 6).cpu(), 0.875, 0.0, mask)
    some = torch.tensor([True, False] * 3).cuda().unsqueeze(1)
    verify(gdn.sample_tokens(logits, u, mask=some), logits, u, mask=some)
    tight = torch.zeros(6, 5001 + 2, dtype=torch.bool, device="cuda")[:, 1:5002]
    tight[:, ::3] = True
    verify(gdn.sample_tokens(logits, u, top_k=50, mask=tight), logits, u, top_k=50, mask=tight)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_rows_at_their_ends(dtype):
    N = 3001
    logits, u, gen = inputs(12, N, dtype, 7)
    low = torch.finfo(dtype).min
    logits[0] = -math.inf                       # nothing to choose
    logits[1, 5] = math.nan
    logits[2, 6] = math.inf
    logits[3] = low                             # the type's lowest value everywhere: all alike
    logits[4, 10:] = low                        # forbidden by that value
    logits[5, :-1] = -math.inf                  # one choice
    logits[6] = torch.finfo(dtype).max / 2      # far from 0, and one less
    logits[6, 7] = low
    heat = torch.ones(12)
    heat[7], heat[8], heat[9], heat[10], heat[11] = -1.0, math.nan, math.inf, 1e-30, 1e30
    got = gdn.sample_tokens(logits, u, heat.cuda(), top_p=0.9)
    tokens, logprobs = (t.cpu() for t in got)
    for b in (0, 1, 2, 7, 8, 9):
        assert tokens[b] == -1 and logprobs[b] == -math.inf
    rows = [3, 4, 5, 6, 10, 11]
    verify((tokens[rows], logprobs[rows]), logits[rows], u[rows], heat[rows], top_p=0.9)
    mask = torch.ones(12, N, dtype=torch.bool)
    mask[1, 5] = mask[2, 6] = False             # what the mask forbids may hold anything
    verify([t[1:3] for t in gdn.sample_tokens(logits, u, mask=mask.cuda())], logits[1:3], u[1:3], mask=mask[1:3])
    for name in ("top_p", "min_p"):
        assert (gdn.sample_tokens(logits[3:6], u[3:6], **{name: math.nan})[0] == -1).all()


@pytest.mark.parametrize("filters", [dict(), dict(top_k=20), dict(top_p=0.9), dict(top_k=2000, top_p=0.99)], ids=str)
def test_random_numbers_at_their_ends(filters):
    """0, the largest below 1, what lies outside and no number."""
    logits, _, _ = inputs(6, 9000, f32, 8)
    logits[:] = logits[0]
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 7.0, -3.0, math.nan]).cuda()
    meant = torch.tensor([0.0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 0.0, 0.0])
    verify(gdn.sample_tokens(logits, u, **filters), logits, meant, **filters)


def test_shares_are_what_is_drawn():
    """Many draws of one row: every token as often as its share says.  A count of n draws of share p is off by more than
    six of its standard deviations once in 10^9."""
    logits, _, gen = inputs(1, 40, f32, 9)
    n = 20000
    u = ((torch.arange(n) + torch.rand(n, generator=gen)) / n).float().clamp(max=1 - 2.0 ** -24).cuda()
    tokens, logprobs = gdn.sample_tokens(logits.expand(n, -1), u)
    p = torch.softmax(logits[0].double().cpu(), 0)
    count = torch.bincount(tokens.cpu().long(), minlength=40).double()
    assert ((count - n * p).abs() <= 6 * (n * p * (1 - p)).sqrt() + 2).all()
    assert torch.allclose(logprobs.cpu().double(), torch.log(p)[tokens.cpu().long()], atol=1e-5)


def test_side_stream_and_graph():
    logits, u, _ = inputs(9, 30000, bf16, 10)
    kinds = dict(temperature=0.9, top_k=300, top_p=0.95)
    want = gdn.sample_tokens(logits, u, **kinds)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = gdn.sample_tokens(logits, u, **kinds)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    kept = logits.clone()
    with torch.cuda.graph(graph):
        got = gdn.sample_tokens(logits, u, **kinds)
    logits.zero_()
    graph.replay()
    torch.cuda.synchronize()
    verify(got, logits, u, **{**kinds})
    logits.copy_(kept)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("seed", range(6))
def test_any(seed):
    """Rows, sizes, spreads and filters at random."""
    gen = torch.Generator().manual_seed(100 + seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi, (1,), generator=gen))  # noqa: E731
    for _ in range(4):
        B, N = pick(1, 40), pick(1, 30000)
        dtype = bf16 if pick(0, 2) else f32
        logits = ((0.1 + 5 * torch.rand(1, generator=gen)) * torch.randn(B, N, generator=gen)).to(dtype)
        u = torch.rand(B, generator=gen)
        heat = 0.2 + 2 * torch.rand(B, generator=gen)
        k = torch.randint(0, 2 * N, (B,), generator=gen).to(torch.int32) if pick(0, 2) else 0
        p = 0.2 + 0.9 * torch.rand(B, generator=gen) if pick(0, 2) else 1.0
        m = 0.3 * torch.rand(B, generator=gen) ** 3 if pick(0, 2) else 0.0
        on = lambda v: v.cuda() if isinstance(v, torch.Tensor) else v  # noqa: E731
        verify(gdn.sample_tokens(logits.cuda(), u.cuda(), heat.cuda(), on(k), on(p), on(m)), logits, u, heat, k, p, m)

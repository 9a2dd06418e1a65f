"""beam_search_step and reorder_states against 64-bit / byte-exact references.

A candidate's score is a sum of three fp32 values (the beam's score, the logit, the normaliser), each off by at
most a few units in the last place at the size of the largest: TOL = 4e-6 at sizes up to 32, measured against
the 64-bit score.  Choices may differ from the 64-bit order only among candidates that close; where the inputs
make scores equal on purpose, they have to be the exact ones."""
import math

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
INF = math.inf


def candidates(logits, scores, finished=None, mask=None):
    """All candidates' scores in 64 bits, [B, W, vocab]; -inf for what may not be chosen."""
    x = logits.cpu().double()
    if mask is not None:
        x = x.masked_fill(~mask.cpu().expand(x.shape), -INF)
    cand = scores.cpu().double().unsqueeze(-1) + torch.log_softmax(x, -1)
    cand = cand.masked_fill(cand.isnan(), -INF)
    if finished is not None:
        f = finished.cpu()
        cand[f] = -INF
        cand[..., 0] = torch.where(f, scores.cpu().double(), cand[..., 0])
    return cand


def verify(got, logits, scores, finished=None, mask=None, n=None, exact=False):
    B, W, vocab = logits.shape
    n = W if n is None else n
    cand = candidates(logits, scores, finished, mask).flatten(1)
    best, flat = torch.sort(cand, dim=1, descending=True, stable=True)
    s, t, p = (y.cpu() for y in got)
    assert s.shape == t.shape == p.shape == (B, n) and t.dtype == p.dtype == torch.int32
    for b in range(B):
        seen = set()
        for j in range(n):
            want = float(best[b, j]) if j < W * vocab else -INF
            score, tok, par = float(s[b, j]), int(t[b, j]), int(p[b, j])
            if want == -INF:
                assert (score, tok, par) == (-INF, -1, j % W), (b, j)
                continue
            tol = 4e-6 * max(1.0, abs(want) / 32)
            assert abs(score - want) <= tol, (b, j, score, want)
            assert 0 <= par < W
            done = finished is not None and bool(finished[b, par])
            assert (tok == -1) == done
            place = par * vocab + (0 if done else tok)
            assert place not in seen
            seen.add(place)
            assert abs(float(cand[b, place]) - want) <= tol
            if exact:
                assert place == int(flat[b, j]), (b, j)


def make(B, W, vocab, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    logits = (4 * torch.randn(B, W, vocab, generator=gen)).to(dtype).cuda()
    return logits, (-10 * torch.rand(B, W, generator=gen)).cuda()


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("B,W,vocab,n", [(1, 1, 1, 1), (2, 3, 1, 3), (1, 4, 32000, 4), (3, 5, 50021, 10), (2, 8, 8191, 16),
                                         (7, 2, 7, 6), (1, 64, 1000, 64), (2, 16, 2049, 33), (1, 1, 1 << 20, 64),
                                         (700, 1, 300, 2), (1, 64, 40000, 64)])
def test_beam(B, W, vocab, n, dtype):
    logits, scores = make(B, W, vocab, dtype, B + W + vocab)
    verify(gdn.beam_search_step(logits, scores, num_candidates=n), logits, scores, n=n)


def test_beam_many_long_rows():
    """More lists than threads in the joining kernel: 64 beams of 2^20 - 1 logits."""
    logits = (4 * torch.randn(1, 64, (1 << 20) - 1, device="cuda", generator=torch.Generator("cuda").manual_seed(1))).to(bf16)
    scores = -torch.arange(64, device="cuda", dtype=f32).unsqueeze(0) / 8
    out, tok, par = (y.cpu() for y in gdn.beam_search_step(logits, scores))
    lse = torch.logsumexp(logits.double(), -1)[0]
    top = torch.topk(logits[0].float(), 64, dim=1)
    cand = (scores[0].double() - lse).unsqueeze(1) + top.values.double()
    best = torch.sort(cand.flatten(), descending=True).values[:64].cpu()
    assert (out[0].double() - best).abs().max() < 8e-6
    picked = logits[0].cpu()[par[0].long(), tok[0].long()].double() + (scores[0].double() - lse).cpu()[par[0].long()]
    assert (picked - best).abs().max() < 8e-6
    assert len({(int(a), int(b)) for a, b in zip(par[0], tok[0])}) == 64


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("kind", ["same", "few", "rising", "falling", "zeros", "one_thread"])
def test_beam_ties_and_orders(kind, dtype):
    """Equal logits go by the lower index, and orders of the input that put every large value in one place."""
    B, W, vocab = 2, 4, 20000
    i = torch.arange(vocab, dtype=f32)
    row = {"same": torch.zeros(vocab), "few": (i * 7919 % 5), "rising": torch.floor(i / 200), "falling": -torch.floor(i / 200),
           "zeros": torch.where(i % 2 == 0, -0.0, 0.0), "one_thread": torch.where(i.long() % 2048 < 8, 9.0, 1.0)}[kind]
    logits = row.expand(B, W, vocab).contiguous().to(dtype).cuda()
    scores = torch.tensor([[-1.0, -1.0, -2.0, -1.0]] * B, device="cuda")
    verify(gdn.beam_search_step(logits, scores, num_candidates=8), logits, scores, n=8, exact=True)
    verify(gdn.beam_search_step(logits, scores, num_candidates=64), logits, scores, n=64, exact=True)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_beam_masks(dtype):
    logits, scores = make(3, 4, 5003, dtype, 3)
    gen = torch.Generator().manual_seed(4)
    mask = (torch.rand(3, 4, 5003, generator=gen) < 0.01).cuda()
    mask[1, 2] = False      # nothing left for one beam
    mask[2] = False         # nothing left for a whole search
    mask[0, 1] = False
    mask[0, 1, 4999] = True  # one token left
    dirty = logits.clone()
    dirty[~mask] = torch.tensor([math.nan, INF, -INF, 1e30], device="cuda").to(dtype).repeat((~mask).sum() // 4 + 1)[:(~mask).sum()]
    got = gdn.beam_search_step(dirty, scores, mask=mask, num_candidates=8)
    verify(got, logits, scores, mask=mask, n=8)
    for shape in ((1, 1, 5003), (3, 1, 5003), (1, 4, 5003), (5003,)):
        m = torch.rand(shape, generator=gen) < 0.3
        verify(gdn.beam_search_step(logits, scores, mask=m.cuda()), logits, scores, mask=m)
    wide = torch.zeros(3, 4, 5010, dtype=torch.bool, device="cuda")  # rows that begin at odd bytes
    wide[..., 3:5006] = mask
    verify(gdn.beam_search_step(logits, scores, mask=wide[..., 3:5006]), logits, scores, mask=mask)


def test_beam_values_that_are_none():
    logits, scores = make(2, 6, 999, f32, 5)
    logits[0, 0, 17] = math.nan
    logits[0, 1, 5] = INF
    logits[0, 2] = -INF
    logits[0, 3, 100:] = -INF
    scores[0, 4] = -INF
    scores[1, 1:] = -INF  # the first step: one beam lives
    clean = logits.clone()
    clean[0, :3] = -INF
    got = gdn.beam_search_step(logits, scores, num_candidates=12)
    verify(got, clean, scores, n=12)
    logits[:] = -INF
    verify(gdn.beam_search_step(logits, scores), logits, scores)
    scores[0, 0] = math.nan
    s, t, p = gdn.beam_search_step(torch.zeros(2, 6, 999, device="cuda"), scores)
    assert 0 not in p[0].tolist()


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_beam_finished(dtype):
    logits, scores = make(4, 5, 4001, dtype, 6)
    finished = torch.zeros(4, 5, dtype=torch.bool, device="cuda")
    finished[0, 2] = finished[1, :] = finished[2, 0] = True
    scores[0, 2], scores[2, 0] = 1.0, -1000.0
    logits[finished] = math.nan
    clean = logits.clone()
    clean[finished] = 0
    verify(gdn.beam_search_step(logits, scores, finished=finished, num_candidates=10), clean, scores, finished=finished, n=10)


def test_beam_layouts_streams_workspace():
    base, scores = make(3, 4, 3003, bf16, 7)
    for off in range(9):  # rows that begin at every place of a 16-byte vector
        wide = torch.zeros(4, 3, 3013, dtype=bf16, device="cuda")
        view = wide[..., off:off + 3003].transpose(0, 1)
        view.copy_(base)
        got = gdn.beam_search_step(view, scores.t().contiguous().t())
        verify(got, base, scores)
    want = gdn.beam_search_step(base, scores)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = gdn.beam_search_step(base, scores, workspace=ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdn.beam_search_step(base, scores)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    strided = base.transpose(1, 2).contiguous().transpose(1, 2)  # the vocabulary is not contiguous: copied
    assert all(torch.equal(a, b) for a, b in zip(gdn.beam_search_step(strided, scores), want))


def test_beam_no_search():
    s, t, p = gdn.beam_search_step(torch.zeros(0, 3, 10, device="cuda"), torch.zeros(0, 3, device="cuda"))
    assert s.shape == t.shape == p.shape == (0, 3)


# ---- states follow ----------------------------------------------------------------------------------


def reordered(states, parents, idx=None):
    B, W = parents.shape
    out = [s.clone() for s in states]
    for b in range(B):
        for i in range(W):
            par = int(parents[b, i])
            src, dst = (b * W + par, b * W + i) if idx is None else (int(idx[b, par]), int(idx[b, i]))
            for o, s in zip(out, states):
                o[dst] = s[src]
    return out


@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 8, 13, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("shape,dtype", [((2, 64, 64), f32), ((3, 1003), bf16), ((5,), torch.uint8), ((1,), torch.float64)])
def test_reorder(W, shape, dtype):
    gen = torch.Generator().manual_seed(W)
    B = 3
    x = (torch.randint(0, 200, (B * W, *shape), generator=gen)).to(dtype)
    parents = torch.randint(0, W, (B, W), generator=gen)
    parents[1] = torch.arange(W).roll(1)  # a cycle: every slot is read after it is wanted elsewhere
    got = x.cuda()
    gdn.reorder_states(got, parents.cuda())
    assert torch.equal(got.cpu(), reordered([x], parents)[0])


def test_reorder_many_tensors_and_a_pool():
    gen = torch.Generator().manual_seed(9)
    B, W, slots = 2, 6, 20
    xs = [torch.randn(slots, 2, 64, 64, generator=gen) for _ in range(40)]
    xs += [torch.randn(slots, 3, 77, generator=gen).to(bf16) for _ in range(40)]
    xs.append(torch.empty(slots, 0))
    idx = torch.randperm(slots, generator=gen)[:B * W].view(B, W)
    parents = torch.randint(0, W, (B, W), generator=gen)
    got = [x.cuda() for x in xs]
    pool = torch.zeros(slots, 2, 2, 64, 64, device="cuda")  # a strided pool: one layer of two
    pool[:, 1] = got[0]
    got[0] = pool[:, 1]
    gdn.reorder_states(got, parents.to(torch.int32).cuda(), state_indices=idx.cuda())
    for a, b in zip(got, reordered(xs, parents, idx)):
        assert torch.equal(a.cpu(), b)
    assert (pool[:, 0] == 0).all()


def test_reorder_places_that_are_none():
    x = torch.arange(8 * 16, dtype=f32).view(8, 16)
    got = x.cuda()
    parents = torch.tensor([[1, -1, 7, 0], [3, 1, 0, 2]], dtype=torch.int32, device="cuda")
    idx = torch.tensor([[0, 1, 2, 3], [4, -1, 6, 9]], dtype=torch.int32, device="cuda")
    gdn.reorder_states(got, parents, state_indices=idx)
    got = got.cpu()
    assert torch.equal(got[0], x[1]) and torch.equal(got[1], x[1])  # followed; negative parent: stays
    assert got[2].isnan().all()                                     # a parent that is no beam
    assert torch.equal(got[3], x[0])
    assert got[4].isnan().all()                                     # its parent's slot is not in the pool
    assert torch.equal(got[6], x[4])                                # beam 2 follows beam 0
    assert torch.equal(got[5], x[5]) and torch.equal(got[7], x[7])


def test_reorder_graph():
    x = torch.randn(8, 4, 64, 64, device="cuda")
    parents = torch.tensor([[1, 0, 3, 2], [0, 0, 1, 1]], dtype=torch.int32, device="cuda")
    want = reordered([x.cpu()], parents.cpu())[0]
    got = x.clone()
    gdn.reorder_states(got, torch.zeros_like(parents) - 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.reorder_states(got, parents)
    assert torch.equal(got, x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), want)

"""beam_search_step on rows of finite logits of any size: the fills that programs put over forbidden or padding tokens,
rows that hold nothing else, rows far from 0.  Against 64 bits, at the tolerance of ``test_gpu_beam.py`` (it grows with
a score's size, beyond 32, as the spacing of fp32 does)."""
import math

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from test_gpu_beam import make, verify

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
FILLS = [-1e4, -1e9, -3e9, -1e10, -1e12, -1e20, -1e30, -1e38, -2.4e38, "min", -math.inf]


def value(fill, dtype):
    return torch.finfo(dtype).min if fill == "min" else fill


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("fill", FILLS, ids=str)
@pytest.mark.parametrize("B,W,vocab", [(1, 4, 32000), (130, 2, 2500), (1, 2, 131072)])
def test_beam_filled_rows(B, W, vocab, fill, dtype):
    """One token in a hundred keeps its logit; in one row only its last, in another only its first."""
    logits, scores = make(B, W, vocab, dtype, 11)
    gen = torch.Generator().manual_seed(12)
    keep = (torch.rand(B, W, vocab, generator=gen) < 0.01).cuda()
    keep[0, 0] = False
    keep[0, 0, vocab - 1] = True
    keep[-1, 1] = False
    keep[-1, 1, 0] = True
    logits[~keep] = value(fill, dtype)
    verify(gdn.beam_search_step(logits, scores, num_candidates=8), logits, scores, n=8)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("fill", FILLS[:-1] + [0.0, 1e9, 1e30, 3e38], ids=str)
def test_beam_rows_of_one_value(fill, dtype):
    """Nothing but the fill: every token has the same share of its beam."""
    scores = torch.tensor([[-2.0, -1.0, -1.5]], device="cuda")
    for vocab in (1, 7, 3001, 70000):
        logits = torch.full((1, 3, vocab), value(fill, dtype), dtype=dtype, device="cuda")
        verify(gdn.beam_search_step(logits, scores, num_candidates=5), logits, scores, n=5, exact=True)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_beam_fills_of_several_kinds(dtype):
    """Fills of different sizes side by side, -inf among them, and a mask over some."""
    logits, scores = make(3, 4, 5003, dtype, 13)
    gen = torch.Generator().manual_seed(14)
    fills = torch.tensor([torch.finfo(dtype).min, -1e30, -math.inf, -1e10, -1e38], dtype=f32).to(dtype).cuda()
    pick = torch.randint(0, 5, (3, 4, 5003), generator=gen).cuda()
    keep = (torch.rand(3, 4, 5003, generator=gen) < 0.02).cuda()
    logits = torch.where(keep, logits, fills[pick])
    verify(gdn.beam_search_step(logits, scores, num_candidates=8), logits, scores, n=8)
    mask = (torch.rand(3, 4, 5003, generator=gen) < 0.5).cuda()
    verify(gdn.beam_search_step(logits, scores, mask=mask, num_candidates=8), logits, scores, mask=mask, n=8)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("offset", [-1e6, -4096.0, 4096.0, 1e6])
def test_beam_rows_far_from_zero(offset, dtype):
    """A constant in front of the logits is none of the softmax's."""
    logits, scores = make(2, 3, 20000, f32, 15)
    logits = (logits + offset).to(dtype)
    verify(gdn.beam_search_step(logits, scores, num_candidates=6), logits, scores, n=6)


def test_beam_largest_logits():
    """Logits up to the largest of the type, rising and falling, so that the running maximum moves all the way."""
    scores = torch.zeros(1, 2, device="cuda")
    for dtype in (bf16, f32):
        top = torch.finfo(dtype).max / 2
        rising = torch.linspace(-top, top, 30011, dtype=torch.float64).to(dtype)
        logits = torch.stack([rising, rising.flip(0)]).unsqueeze(0).cuda()
        logits[..., 5:900] = torch.randn(895, device="cuda").to(dtype)
        verify(gdn.beam_search_step(logits, scores, num_candidates=3), logits, scores, n=3)

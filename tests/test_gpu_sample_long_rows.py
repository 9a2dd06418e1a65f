"""Sampling from the longest vocabularies: sums of a slice's equal shares hold whatever the shares' bits and the row's
alignment."""
import math

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from test_gpu_sample import verify

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
N = 1 << 20


def equal_row(dtype, bits, offset):
    """Rows [3, N], `offset` elements behind 16-byte boundaries, of one best logit and equal ones 8 below it, and a
    temperature at which an equal one's share of 2^42 lies 2^14 below 2^bits: all ones from bit 15 on."""
    wide = torch.zeros(3, N + 16, dtype=dtype, device="cuda")
    logits = wide[:, offset:offset + N]
    logits[:, 5] = 8.0
    heat = torch.tensor(8 / (42 * math.log(2) - math.log(2.0 ** bits - 2.0 ** 14)), dtype=f32).item()
    share = 2.0 ** 42 * math.exp(-8 / heat)
    assert 2.0 ** bits - 0.9 * 2 ** 15 < share < 2.0 ** bits - 0.1 * 2 ** 15
    return logits, heat


@pytest.mark.parametrize("filters", [dict(top_p=0.5), dict(top_k=1000003, top_p=0.5), dict(top_p=0.5, min_p=1e-4)], ids=str)
@pytest.mark.parametrize("bits", [30, 31])
@pytest.mark.parametrize("dtype,offset", [(bf16, 1), (bf16, 0), (bf16, 7), (f32, 1)])
def test_shares_of_full_parts(dtype, offset, bits, filters):
    logits, heat = equal_row(dtype, bits, offset)
    u = torch.tensor([0.1, 0.5001, 0.9]).cuda()
    verify(gdn.sample_tokens(logits, u, temperature=heat, **filters), logits, u, temperature=heat, **filters)


@pytest.mark.parametrize("dtype,offset", [(bf16, 1), (f32, 3)])
def test_random_rows_off_their_boundaries(dtype, offset):
    gen = torch.Generator().manual_seed(4)
    wide = (2 * torch.randn(2, N + 16, generator=gen)).to(dtype).cuda()
    logits, u = wide[:, offset:offset + N], torch.rand(2, generator=gen).cuda()
    for filters in (dict(top_p=0.95), dict(temperature=1.2, top_k=2000, top_p=0.9, min_p=0.001)):
        verify(gdn.sample_tokens(logits, u, **filters), logits, u, **filters)

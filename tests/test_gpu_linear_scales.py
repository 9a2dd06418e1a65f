"""Linear attention where sizes differ by orders of magnitude: what has decayed leaves nothing of its size behind.

A state X that a chunk of n tokens moves on by l^n X + U has to come out as U to U's own precision wherever l^n X is small
beside it, however large X was.  Tolerances are those of test_gpu_linear.py, held by every row of every head by itself, so
that a large one lends nothing to its neighbours: fp32 1e-5 * RMS, bf16 2e-3 * RMS before the rounding, states 1e-5 * RMS.

A row's terms may cancel: where one token is left, o = scale (q . k) v, and q . k may be all but 0 while its products are
not.  So a row may be off by what its terms are rounded by too.  With A the sum of their absolute values (the same formulas
with every input's absolute value):
  fp32: an element meets some 200 roundings, 128 of a product over the width, 64 over the chunk and a few, each of 2^-24 of a
    partial sum of A at most, 2^-24 / sqrt(3) on average: six standard deviations are 6 * sqrt(200) * 2^-24 / sqrt(3) = 3e-6 A;
  bf16: a term has one operand of two bf16 parts, off by 2^-17 of itself, and fp32 sums as above: 2^-16 A."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from parity import BF16_TOL, FP32_TOL, half_ulp_bf16
from test_gpu_linear import call, make, packed_case, reference, verify

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
DECAYS = [-float("inf"), -60.0, -1.0, -0.05]


def verify_rows(name, got, ref, size, dtype):
    """Every row [width] by itself; size: its terms' absolute values, summed."""
    assert got.dtype == dtype and got.shape == ref.shape
    a, b = got.detach().double().cpu(), ref.cpu()
    bound = (FP32_TOL if dtype == f32 else BF16_TOL) * b.square().mean(-1, keepdim=True).sqrt().expand_as(b)
    bound = bound + (3e-6 if dtype == f32 else 2.0 ** -16) * size.cpu()
    if dtype == bf16:
        bound = bound + torch.from_numpy(half_ulp_bf16(torch.maximum(a.abs(), b.abs()).numpy()))
    over = (a - b).abs() - bound
    assert a.isfinite().all() and over.max() <= 0, (name, [int(i) for i in torch.unravel_index(over.argmax(), over.shape)], float(over.max()))


def compare(x, dtype, cu=None, spans=None):
    o, ht = call(x, cu_seqlens=cu)
    grads = gdn.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dht"], initial_state=x["h0"], cu_seqlens=cu)
    ref = reference(x, spans, backward=True)
    size = reference(dict(x, **{n: x[n].abs() for n in ("q", "k", "v", "do", "h0", "dht")}), spans, backward=True)
    for name, got in zip(("o", "dq", "dk", "dv"), (o,) + grads[:3]):
        verify_rows(name, got, ref[name], size[name], dtype)
    for name, got in (("ht", ht), ("dh0", grads[3])):
        for n in range(got.shape[0]):
            for h in range(got.shape[1]):
                verify(name, got[n, h], ref[name][n, h], dtype)


@pytest.mark.parametrize("size", [1e3, 1e6])
@pytest.mark.parametrize("T", [64, 70, 1000, 2000])  # one chunk, two, whole and in segments
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_large_states(dtype, T, size):
    x = make(1, T, 4, 4, 128, 128, dtype, seed=T)
    x["g"] = torch.tensor(DECAYS, device="cuda")
    x["h0"] *= size
    x["dht"] *= size
    compare(x, dtype)


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_large_states_of_other_widths(dtype, K, V):
    x = make(2, 200, 2, 4, K, V, dtype, seed=K + V)
    x["g"] = torch.tensor(DECAYS, device="cuda")
    x["h0"] *= 1e6
    x["dht"] *= 1e6
    compare(x, dtype)


@pytest.mark.parametrize("T", [128, 1400])
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_one_large_token(dtype, T):
    """Near the end of a chunk in the order of each scan, so that it fills the state that the next chunk begins with."""
    x = make(1, T, 4, 4, 128, 128, dtype, seed=T + 1)
    x["g"] = torch.tensor(DECAYS, device="cuda")
    for at in (60, T - 61):
        for name in ("q", "k", "v", "do"):
            x[name][:, at] *= 1e3
    compare(x, dtype)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_large_states_of_packed_sequences(dtype):
    x, cu, spans = packed_case([64, 3000, 0, 1, 200, 65], 4, 4, 64, 64, dtype, seed=3)
    x["g"] = torch.tensor(DECAYS, device="cuda")
    x["h0"] *= 1e6
    x["dht"] *= 1e6
    compare(x, dtype, cu, spans)


@pytest.mark.parametrize("Hv", [2, 160])  # in segments and whole
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_slow_decay_over_many_chunks(dtype, Hv):
    """300 chunks that add nothing, with a decay of a chunk that lies between two fp32 numbers: rounded to one of them alone it
    would be off by 300 * 2^-25 = 9e-6 in the end.  What may be off: 300 roundings of the state, by 2^-24 / sqrt(3) of itself
    on average, of which six standard deviations are 6 * sqrt(300 / 3) * 2^-24 = 3.6e-6."""
    T, K, V = 300 * 64, 64, 64
    g = torch.full((Hv,), -1073.5 * 2.0 ** -24 / 64, device="cuda")
    q, v = torch.zeros(1, T, 1, K, dtype=dtype, device="cuda"), torch.zeros(1, T, Hv, V, dtype=dtype, device="cuda")
    h0 = torch.randn(1, Hv, K, V, generator=torch.Generator().manual_seed(1)).cuda()
    _, ht = gdn.chunk_linear_attention(q, q, v, g, initial_state=h0, output_final_state=True)
    want = h0.double() * torch.exp(g.double() * T)[:, None, None]
    assert (ht.double() / want - 1).abs().max() < 3.7e-6
    _, _, _, dh0 = gdn.chunk_linear_attention_bwd(q, q, v, g, v, h0, initial_state=h0)
    assert torch.equal(dh0, ht)

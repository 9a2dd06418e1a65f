"""Linear attention: what one sequence holds does not reach another, in the gradients either, and the same call gives the
same bits."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from test_gpu_linear import call, make, packed_case, reference, verify

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
NAMES = ("o", "ht", "dq", "dk", "dv", "dh0")


def everything(x, cu=None):
    back = gdn.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], x["dht"], initial_state=x["h0"], cu_seqlens=cu)
    return dict(zip(NAMES, call(x, cu_seqlens=cu) + back))


PACKED = [  # lengths, the sequences that are spoilt, Hq, Hv, K, V
    ([70, 130, 61], [1], 1, 2, 128, 128), ([5, 9, 1, 30, 64, 0, 3], [1, 3], 2, 2, 64, 128), ([63, 1, 64, 65], [0, 2], 1, 3, 128, 64),
    ([3000, 40, 500], [1], 2, 2, 64, 64), ([40, 3000, 500], [1], 1, 2, 128, 128), ([2, 1] * 20, [0, 7, 39], 1, 2, 64, 64),
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: "%d_%s" % (len(c[0]), "_".join(map(str, c[2:]))))
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_packed_neighbours_of_what_is_not_finite(dtype, case):
    lengths, bad, Hq, Hv, K, V = case
    x, cu, spans = packed_case(lengths, Hq, Hv, K, V, dtype, seed=len(lengths))
    clean = {n: t.clone() for n, t in everything(x, cu).items()}
    keep = torch.ones(sum(lengths), dtype=torch.bool, device="cuda")
    for n in bad:
        _, lo, hi = spans[n]
        keep[lo:hi] = False
        for name in ("q", "k", "v", "do"):
            x[name][0, lo:hi] = float("nan")
            x[name][0, lo] = float("inf")
        x["h0"][n] = float("nan")
        x["dht"][n] = float("inf")
    got = everything(x, cu)
    for name in ("o", "dq", "dk", "dv"):
        assert clean[name].isfinite().all() and torch.equal(got[name][0, keep], clean[name][0, keep])
        assert got[name][0, ~keep].isnan().any()
    for name in ("ht", "dh0"):
        for n in range(len(lengths)):
            assert not got[name][n].isfinite().any() if n in bad else torch.equal(got[name][n], clean[name][n])


@pytest.mark.parametrize("T", [30, 100, 1500])
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_rows_beside_what_is_not_finite(dtype, T):
    x = make(3, T, 1, 2, 128, 128, dtype, seed=T)
    clean = {n: t.clone() for n, t in everything(x).items()}
    for name in ("q", "k", "v", "do", "h0", "dht"):
        x[name][1] = float("nan")
    got = everything(x)
    for name in NAMES:
        assert torch.equal(got[name][::2], clean[name][::2]) and got[name][1].isnan().all()


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_gradients_where_offsets_leave_rows_out(dtype):
    """Offsets that begin late, end early, fall or leave the tokens: the claimed rows have their gradients, the others 0."""
    T = 400
    x = make(1, T, 2, 4, 128, 128, dtype, seed=11, h0=False)
    cu = torch.tensor([7, 90, 90, 250, T + 5, T + 5, 300, 390], device="cuda")
    spans = [(0, 7, 90), (0, 0, 0), (0, 90, 250), (0, 0, 0), (0, 0, 0), (0, 0, 0), (0, 300, 390)]
    gen = torch.Generator().manual_seed(2)
    x["h0"], x["dht"] = (torch.randn(7, 4, 128, 128, generator=gen).cuda() for _ in range(2))
    got, ref = everything(x, cu), reference(x, spans, backward=True)
    for name in NAMES:
        verify(name, got[name], ref[name], dtype)
    for name in ("o", "dq", "dk", "dv"):
        for lo, hi in ((0, 7), (250, 300), (390, T)):
            assert (got[name][0, lo:hi] == 0).all()


CASES = [(1, 97, 32, 32, 128, 128), (4, 500, 4, 8, 128, 128), (1, 5000, 2, 4, 128, 128), (1, 777, 8, 8, 64, 128), (2, 1000, 4, 8, 64, 64)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_the_same_call_gives_the_same_bits(dtype, case):
    x = make(*case, dtype, seed=sum(case))
    first = {n: t.clone() for n, t in everything(x).items()}
    for _ in range(10):
        again = everything(x)
        assert all(torch.equal(again[n], first[n]) for n in NAMES)

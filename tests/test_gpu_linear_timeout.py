"""Linear attention's bounded waits, exercised in the permitted form: a load that every CTA skips (gdn_debug_set_wait), so that
one wait cannot complete.  The kernel gives up after its second, what it concerns is NaN, and the next call is the one before.
The limit is the kernel's own: one that is passed in costs it registers, and 3 to 13 % of its time."""
import contextlib

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from test_gpu_linear import make, packed_case
from test_gpu_linear_neighbours import NAMES, everything

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


@contextlib.contextmanager
def skipped(chunk):
    lib = gdn.load_library()
    lib.gdn_debug_set_wait(0, chunk)
    try:
        yield
        torch.cuda.synchronize()
    finally:
        lib.gdn_debug_set_wait(0, -1)


@pytest.mark.parametrize("T,Hv,chunk", [(300, 4, 1), (300, 4, 4), (20000, 8, 1)])
def test_what_a_skipped_load_concerns(T, Hv, chunk):
    """Whole sequences, their last, short chunk among them, and segments."""
    x = make(2 if T < 1000 else 1, T, 2, Hv, 128, 128, bf16, seed=T + chunk)
    clean = {n: t.clone() for n, t in everything(x).items()}
    with skipped(chunk):
        got = everything(x)
    assert all(got[n].isnan().all() for n in NAMES)
    again = everything(x)
    assert all(torch.equal(again[n], clean[n]) for n in NAMES)


@pytest.mark.parametrize("K,V", [(64, 128)])
def test_sequences_without_such_a_chunk(K, V):  # enough heads that none is cut
    x, cu, spans = packed_case([300, 50, 0, 64], 8, 16, K, V, bf16, seed=4)
    clean = {n: t.clone() for n, t in everything(x, cu).items()}
    with skipped(1):
        got = everything(x, cu)
    for name in ("o", "dq", "dk", "dv"):
        assert got[name][0, :300].isnan().all() and torch.equal(got[name][0, 300:], clean[name][0, 300:])
    for name in ("ht", "dh0"):
        assert got[name][0].isnan().all() and torch.equal(got[name][1:], clean[name][1:])
    again = everything(x, cu)
    assert all(torch.equal(again[n], clean[n]) for n in NAMES)

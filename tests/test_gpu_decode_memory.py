"""A decoding call that finds no memory for its output raises what PyTorch raises, and the next call works."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn

pytestmark = pytest.mark.gpu


def test_out_of_memory():
    T = 2 ** 30  # half a terabyte of o; the inputs repeat one token
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    a = dict(q=x.expand(1, T, 1, 64), k=x.expand(1, T, 1, 64), v=x.expand(1, T, 4, 64), g=torch.zeros(1, 1, 1, device="cuda").expand(1, T, 4),
             beta=torch.zeros(1, 1, 1, device="cuda").expand(1, T, 4), state=torch.ones(1, 4, 64, 64, device="cuda"))
    with pytest.raises(torch.cuda.OutOfMemoryError):
        gdn.recurrent_gated_delta_rule(**a)
    assert (a["state"] == 1).all()
    few = {n: (y if n == "state" else y[:, :2]) for n, y in a.items()}
    assert (gdn.recurrent_gated_delta_rule(**few) == 0).all()

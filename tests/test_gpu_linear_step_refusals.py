"""What the step of linear attention refuses, and with which error."""
import pytest
import torch

import gated_delta_rule_50_gb300 as gdn
from test_linear_refusals import chunk_args

pytestmark = pytest.mark.gpu
BAD = {
    "g per token": (lambda a: a.update(g=torch.zeros(2, 3, 4, device="cuda")), ValueError),
    "g shape": (lambda a: a.update(g=a["g"][:2]), ValueError),
    "g complex": (lambda a: a.update(g=a["g"].to(torch.complex64)), TypeError),
    "g on the host": (lambda a: a.update(g=a["g"].cpu()), ValueError),
    "mixed dtypes": (lambda a: a.update(v=a["v"].float()), TypeError),
    "state dtype": (lambda a: a.update(state=a["state"].to(torch.bfloat16)), TypeError),
    "state shape": (lambda a: a.update(state=a["state"][..., :32]), ValueError),
    "widths": (lambda a: a.update(step_args(K=96)), gdn.GdnError),
}


def step_args(**kw):
    a = chunk_args("cuda", **kw)
    a["state"] = a.pop("initial_state")
    return a


@pytest.mark.parametrize("name", list(BAD))
def test_refusals(name):
    a = step_args()
    change, error = BAD[name]
    change(a)
    with pytest.raises(error):
        gdn.recurrent_linear_attention(**a)

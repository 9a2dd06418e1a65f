"""What linear attention and the sampling of tokens refuse, and with which error; nothing here reaches a kernel."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
bf16, f32 = torch.bfloat16, torch.float32


def chunk_args(device="cpu", dtype=bf16, B=2, T=3, Hq=2, Hv=4, K=64, V=64):
    def mk(*s, dt=dtype):
        return torch.zeros(*s, dtype=dt, device=device)

    return dict(q=mk(B, T, Hq, K), k=mk(B, T, Hq, K), v=mk(B, T, Hv, V), g=mk(Hv, dt=f32), initial_state=mk(B, Hv, K, V, dt=f32))


def sample_args(device="cpu", B=2, N=10):
    return dict(logits=torch.zeros(B, N, device=device), random=torch.zeros(B, device=device))


def test_not_tensors():
    a = chunk_args()
    for name in ("q", "k", "v", "g", "initial_state"):
        with pytest.raises((TypeError, AttributeError), match="tensor|requires_grad"):
            gdn.chunk_linear_attention(**dict(a, **{name: 1.0}))
        with pytest.raises(TypeError, match="tensor"):
            gdn.chunk_linear_attention_fwd(**dict(a, **{name: 1.0}))
    with pytest.raises(TypeError, match="tensor"):
        gdn.recurrent_linear_attention(a["q"], a["k"], a["v"], 0.5, a["initial_state"])
    with pytest.raises(TypeError, match="tensor"):
        gdn.sample_tokens([[1.0]], torch.zeros(1))


def test_no_cpu_path():
    a = chunk_args()
    with pytest.raises(ValueError, match="CUDA"):
        gdn.chunk_linear_attention(**a)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.chunk_linear_attention_bwd(a["q"], a["k"], a["v"], a["g"], a["v"])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.recurrent_linear_attention(a["q"], a["k"], a["v"], a["g"], a["initial_state"])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.sample_tokens(**sample_args())


def test_the_decay_has_no_gradient():
    a = chunk_args()
    a["g"].requires_grad_()
    with pytest.raises(ValueError, match="constant"):
        gdn.chunk_linear_attention(**a)


BAD = {
    "k shape": (lambda a: a.update(k=a["k"][:, :2]), ValueError),
    "v shape": (lambda a: a.update(v=a["v"][:1]), ValueError),
    "g per token": (lambda a: a.update(g=torch.zeros(2, 3, 4, device="cuda")), ValueError),
    "g shape": (lambda a: a.update(g=a["g"][:2]), ValueError),
    "g complex": (lambda a: a.update(g=a["g"].to(torch.complex64)), TypeError),
    "g on the host": (lambda a: a.update(g=a["g"].cpu()), ValueError),
    "mixed dtypes": (lambda a: a.update(v=a["v"].float()), TypeError),
    "half": (lambda a: a.update(q=a["q"].half(), k=a["k"].half(), v=a["v"].half()), TypeError),
    "three dimensions": (lambda a: a.update(q=a["q"][0], k=a["k"][0]), ValueError),
    "state dtype": (lambda a: a.update(initial_state=a["initial_state"].to(bf16)), TypeError),
    "state shape": (lambda a: a.update(initial_state=a["initial_state"][:1]), ValueError),
    "offsets with a batch": (lambda a: a.update(cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
    "offsets' dtype": (lambda a: a.update({k: v[:1] for k, v in a.items() if k != "g"}, cu_seqlens=torch.zeros(2, device="cuda")), TypeError),
    "offsets on the host": (lambda a: a.update({k: v[:1] for k, v in a.items() if k != "g"}, cu_seqlens=torch.zeros(2, dtype=torch.int32)), ValueError),
    "no offsets": (lambda a: a.update({k: v[:1] for k, v in a.items() if k != "g"}, cu_seqlens=torch.zeros(0, dtype=torch.int32, device="cuda")), ValueError),
    "widths": (lambda a: a.update(chunk_args("cuda", K=96)), gdn.GdnError),
    "heads": (lambda a: a.update(chunk_args("cuda", Hq=3)), gdn.GdnError),
    "scale": (lambda a: a.update(scale="x"), TypeError),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(BAD))
def test_chunk_refusals(name):
    a = chunk_args("cuda")
    change, error = BAD[name]
    change(a)
    with pytest.raises(error):
        gdn.chunk_linear_attention(**a)


@pytest.mark.gpu
def test_derivatives_are_not_dropped():
    a = chunk_args("cuda")
    a["v"].requires_grad_()
    with pytest.raises(ValueError, match="chunk_linear_attention"):
        gdn.chunk_linear_attention_fwd(**a)
    with pytest.raises(ValueError, match="no backward"):
        gdn.recurrent_linear_attention(a["q"], a["k"], a["v"], a["g"], a["initial_state"])
    o, _ = gdn.chunk_linear_attention(**a)
    (g,) = torch.autograd.grad(o.float().sum(), a["v"], create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.float().sum(), a["v"])
    import torch.autograd.forward_ad as fwAD
    with fwAD.dual_level(), torch.no_grad():
        v = fwAD.make_dual(a["v"].detach(), torch.ones_like(a["v"]))
        with pytest.raises(ValueError, match="tangents"):
            gdn.chunk_linear_attention(a["q"], a["k"], v, a["g"])
    s = sample_args("cuda")
    s["logits"].requires_grad_()
    with pytest.raises(ValueError, match="no backward"):
        gdn.sample_tokens(**s)


@pytest.mark.gpu
@pytest.mark.parametrize("change,error", [
    (dict(logits=torch.zeros(2, 3, 4)), ValueError), (dict(logits=torch.zeros(2, 10).half()), TypeError),
    (dict(random=torch.zeros(3)), ValueError), (dict(random=torch.zeros(2).double()), TypeError), (dict(logits=torch.zeros(2, 0)), ValueError),
    (dict(top_k=torch.zeros(2)), TypeError), (dict(top_k=torch.zeros(3, dtype=torch.int32)), ValueError), (dict(top_k=1.5), TypeError),
    (dict(top_p=torch.zeros(2, dtype=torch.int32)), TypeError), (dict(temperature="hot"), TypeError), (dict(min_p=torch.zeros(1)), ValueError),
    (dict(mask=torch.ones(2, 10)), TypeError), (dict(mask=torch.ones(3, 10, dtype=torch.bool)), ValueError),
    (dict(logits=torch.zeros(1, (1 << 20) + 1), random=torch.zeros(1)), ValueError)], ids=lambda x: None)
def test_sample_refusals(change, error):
    a = sample_args("cuda")
    a.update({k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in change.items()})
    with pytest.raises(error):
        gdn.sample_tokens(**a)
    with pytest.raises(ValueError, match="must be on"):
        gdn.sample_tokens(torch.zeros(2, 10, device="cuda"), torch.zeros(2))


# The entry points in C, in a process that sees no GPU: what is refused returns before anything is launched.
_STATUSES = r"""
import ctypes as C
import gated_delta_rule_50_gb300 as gdn
lib = gdn.load_library()
class S(C.Structure): _fields_ = [(n, C.c_int64) for n in ("batch", "token", "head")]
class P(C.Structure): _fields_ = ([(n, C.c_int64) for n in ("B", "T", "Hq", "Hv", "K", "V", "n_seqs")] + [("cu", C.c_void_p), ("io", C.c_int),
                                  ("scale", C.c_float)] + [(n, S) for n in ("q", "k", "v", "d_o")])
class Q(C.Structure): _fields_ = ([(n, C.c_int64) for n in ("B", "vocab", "logits_row", "mask_row")] + [("dtype", C.c_int)] +
                                  [(n, C.c_void_p) for n in ("temperatures", "top_ps", "min_ps", "top_ks")] +
                                  [(n, C.c_float) for n in ("temperature", "top_p", "min_p")] + [("top_k", C.c_int32)])
def prob(**kw):
    p = P(1, 128, 2, 4, 128, 128, 1, None, 1, 0.1)
    for n, v in kw.items(): setattr(p, n, v)
    return p
for f in ("fwd", "bwd"):
    fn = getattr(lib, "gdn_linear_%s_workspace_bytes" % f); fn.restype = C.c_size_t
    for kw, ok in (({}, 1), (dict(Hv=3), 0), (dict(K=96), 0), (dict(io=7), 0), (dict(n_seqs=2), 0), (dict(T=0), 1), (dict(B=0, n_seqs=0), 1),
                   (dict(B=2, n_seqs=3, cu=16), 0), (dict(T=-1), 0), (dict(Hv=1 << 15, Hq=1), 0), (dict(B=1 << 20, n_seqs=1 << 20, T=1 << 12), 0)):
        assert (fn(C.byref(prob(**kw))) > 0) == bool(ok), (f, kw)
    assert fn(None) == 0
x, odd = C.c_void_p(4096), C.c_void_p(4097)
def fwd(p, q=x, k=x, v=x, g=x, h0=x, o=x, ht=x, ws=x, n=1 << 40):
    return lib.gdn_linear_fwd(p if p is None else C.byref(p), q, k, v, g, h0, o, ht, ws, C.c_size_t(n), None)
assert fwd(None) == 1 and fwd(prob(), q=None) == 1 and fwd(prob(), o=None) == 1 and fwd(prob(), o=C.c_void_p(4104)) == 1
assert fwd(prob(), v=odd) == 1 and fwd(prob(), h0=C.c_void_p(4100)) == 1 and fwd(prob(), g=odd) == 1 and fwd(prob(cu=4097)) == 1
assert fwd(prob(K=32)) == 2 and fwd(prob(), ws=None) == 3 and fwd(prob(), n=16) == 3 and fwd(prob(), ws=C.c_void_p(4112)) == 3
def bwd(p, q=x, do=x, dht=x, dq=x, dk=x, dv=x, dh0=x, ws=x, n=1 << 40):
    return lib.gdn_linear_bwd(C.byref(p), q, x, x, x, x, do, dht, dq, dk, dv, dh0, ws, C.c_size_t(n), None)
assert bwd(prob(), q=None) == 1 and bwd(prob(), do=None) == 1 and bwd(prob(), dq=C.c_void_p(4104)) == 1 and bwd(prob(), dh0=odd) == 1
assert bwd(prob(), ws=None) == 3 and bwd(prob(), n=16) == 3 and bwd(prob(V=32)) == 2
def sample(p, logits=x, u=x, tokens=x, logprobs=x):
    return lib.gdn_sample(p if p is None else C.byref(p), logits, u, None, tokens, logprobs, None)
def sp(**kw):
    p = Q(2, 100, 100, 0, 1)
    for n, v in kw.items(): setattr(p, n, v)
    return p
assert sample(None) == 1 and sample(sp(B=-1)) == 1 and sample(sp(vocab=0)) == 1 and sample(sp(dtype=5)) == 1 and sample(sp(vocab=(1 << 20) + 1)) == 2
assert sample(sp(B=0)) == 0 and sample(sp(), logits=None) == 1 and sample(sp(), tokens=odd) == 1 and sample(sp(), logits=odd) == 1 and sample(sp(top_ks=4097)) == 1
assert lib.gdn_linear_recurrent(None, x, x, x, x, x, None, x, None) == 1
print("as expected")
"""


def test_statuses_in_c():
    r = subprocess.run([sys.executable, "-c", _STATUSES], capture_output=True, text=True, cwd=ROOT,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT))
    assert r.returncode == 0 and "as expected" in r.stdout, r.stdout + r.stderr

"""What the decoding calls refuse, and with which error; nothing here reaches a kernel."""
import os
import struct
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_50_gb300 as gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def step_args(device="cpu", dtype=torch.bfloat16, B=2, T=1, Hq=2, Hv=4, K=64, V=64, slots=3):
    mk = lambda *s, dt=dtype: torch.zeros(*s, dtype=dt, device=device)
    return dict(q=mk(B, T, Hq, K), k=mk(B, T, Hq, K), v=mk(B, T, Hv, V), g=mk(B, T, Hv, dt=torch.float32),
                beta=mk(B, T, Hv, dt=torch.float32), state=mk(slots, Hv, K, V, dt=torch.float32))


def test_not_tensors():
    a = step_args()
    for name in ("k", "v", "g", "beta", "state"):
        with pytest.raises(TypeError, match="tensor"):
            gdn.recurrent_gated_delta_rule(**dict(a, **{name: 1.0}))
    with pytest.raises(TypeError, match="tensor"):
        gdn.beam_search_step([[1.0]], torch.zeros(1, 1))
    with pytest.raises(TypeError):
        gdn.reorder_states(3, torch.zeros(1, 1))
    with pytest.raises(TypeError, match="tensor"):
        gdn.reorder_states([None], torch.zeros(1, 1))


def test_no_cpu_path():
    a = step_args()
    with pytest.raises(ValueError, match="CUDA"):
        gdn.recurrent_gated_delta_rule(**a)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.tree_gated_delta_rule(a["q"], a["k"], a["v"], a["g"], a["beta"], torch.zeros(2, 1, dtype=torch.int32), a["state"])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.beam_search_step(torch.zeros(1, 2, 5), torch.zeros(1, 2))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.reorder_states(torch.zeros(4, 2), torch.zeros(2, 2, dtype=torch.int32))


BAD_STEP = {
    "q shape": (lambda a: a.update(q=a["q"][:, :, :1]), ValueError),
    "v shape": (lambda a: a.update(v=a["v"][:1]), ValueError),
    "g shape": (lambda a: a.update(g=a["g"][..., :1]), ValueError),
    "mixed dtypes": (lambda a: a.update(v=a["v"].float()), TypeError),
    "half": (lambda a: a.update(q=a["q"].half(), k=a["k"].half(), v=a["v"].half()), TypeError),
    "state dtype": (lambda a: a.update(state=a["state"].to(torch.bfloat16)), TypeError),
    "state shape": (lambda a: a.update(state=a["state"][:, :2]), ValueError),
    "state layout": (lambda a: a.update(state=a["state"].transpose(2, 3)), ValueError),
    "too few slots": (lambda a: a.update(state=a["state"][:1]), gdn.GdnError),
    "shared slots in place": (lambda a: a.update(state=a["state"][:1].expand(3, -1, -1, -1)), gdn.GdnError),
    "index count": (lambda a: a.update(state_indices=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
    "index dtype": (lambda a: a.update(state_indices=torch.zeros(2, device="cuda")), TypeError),
    "cpu index": (lambda a: a.update(state_indices=torch.zeros(2, dtype=torch.int32)), ValueError),
    "cu with batch": (lambda a: a.update(cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
    "token rows": (lambda a: a.update(token_indices=torch.zeros(1, 4, dtype=torch.int32, device="cuda")), ValueError),
    "out shape": (lambda a: a.update(out_state=a["state"].clone()), ValueError),
    "out overlaps": (lambda a: a.update(out_state=a["state"][1:]), gdn.GdnError),
    "gradient": (lambda a: a.update(v=a["v"].requires_grad_()), ValueError),
    "widths": (lambda a: a.update(step_args("cuda", K=96, V=64)), gdn.GdnError),
    "heads": (lambda a: a.update(step_args("cuda", Hq=3, Hv=4)), gdn.GdnError),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(BAD_STEP))
def test_recurrent_refusals(name):
    a = step_args("cuda")
    change, error = BAD_STEP[name]
    change(a)
    before = a["state"].clone()
    with pytest.raises(error):
        gdn.recurrent_gated_delta_rule(**a)
    assert torch.equal(a["state"], before)


@pytest.mark.gpu
def test_tree_refusals():
    a = step_args("cuda", T=4)
    call = lambda p, **kw: gdn.tree_gated_delta_rule(*[dict(a, **kw)[n] for n in ("q", "k", "v", "g", "beta")], p, a["state"])
    ok = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    call(ok)
    with pytest.raises(ValueError):
        call(ok[:, :3])
    with pytest.raises(TypeError):
        call(ok.float())
    with pytest.raises(ValueError):
        call(ok, q=None)
    b = step_args("cuda", T=65)
    with pytest.raises(gdn.GdnError) as e:
        gdn.tree_gated_delta_rule(b["q"], b["k"], b["v"], b["g"], b["beta"],
                                  torch.full((2, 65), -1, dtype=torch.int32, device="cuda"), b["state"])
    assert e.value.status == 2


@pytest.mark.gpu
def test_beam_refusals():
    x, s = torch.zeros(2, 3, 50, device="cuda"), torch.zeros(2, 3, device="cuda")
    for kw, error in ((dict(num_candidates=0), ValueError), (dict(num_candidates=65), ValueError),
                      (dict(finished=torch.zeros(2, 2, dtype=torch.bool, device="cuda")), ValueError),
                      (dict(finished=torch.zeros(2, 3, device="cuda")), TypeError),
                      (dict(mask=torch.zeros(2, 3, 50, device="cuda")), TypeError),
                      (dict(mask=torch.zeros(2, 3, 49, dtype=torch.bool, device="cuda")), ValueError),
                      (dict(mask=torch.zeros(2, 3, 50, dtype=torch.bool)), ValueError)):
        with pytest.raises(error):
            gdn.beam_search_step(x, s, **kw)
    with pytest.raises(ValueError):
        gdn.beam_search_step(x[0], s)
    with pytest.raises(TypeError):
        gdn.beam_search_step(x.half(), s)
    with pytest.raises(TypeError):
        gdn.beam_search_step(x, s.double())
    with pytest.raises(ValueError):
        gdn.beam_search_step(x, s[:, :2])
    with pytest.raises(ValueError):
        gdn.beam_search_step(torch.zeros(1, 65, 2, device="cuda"), torch.zeros(1, 65, device="cuda"))
    with pytest.raises(gdn.GdnError):
        gdn.beam_search_step(torch.zeros(1, 1, (1 << 20) + 1, device="cuda"), torch.zeros(1, 1, device="cuda"))
    with pytest.raises(gdn.GdnError):
        gdn.beam_search_step(torch.zeros(1, 1, 0, device="cuda"), torch.zeros(1, 1, device="cuda"))


@pytest.mark.gpu
def test_reorder_refusals():
    x, p = torch.zeros(6, 8, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    gdn.reorder_states([], p)
    with pytest.raises(ValueError):
        gdn.reorder_states(x, p[0])
    with pytest.raises(ValueError):
        gdn.reorder_states([x, torch.zeros(5, 8, device="cuda")], p)
    with pytest.raises(ValueError):
        gdn.reorder_states(torch.zeros(6, 4, 8, device="cuda").transpose(1, 2), p)
    with pytest.raises(ValueError):
        gdn.reorder_states([x, torch.zeros(6, 8)], p)
    with pytest.raises(ValueError):
        gdn.reorder_states(x, p, state_indices=p[:1])
    with pytest.raises(TypeError):
        gdn.reorder_states(x, p.float())
    with pytest.raises(ValueError):
        gdn.reorder_states(torch.zeros(65, 1, device="cuda"), torch.zeros(1, 65, dtype=torch.int32, device="cuda"))
    with pytest.raises(gdn.GdnError):
        gdn.reorder_states(x[:5], p)
    with pytest.raises(gdn.GdnError):
        gdn.reorder_states(x[:1].expand(6, 8), p)


# The C entries with placeholder addresses, in a child process that sees no GPU: a launch could only fail.
# gdn_decode_problem, gdn_beam_problem and gdn_state_view, packed as the C compiler lays them out
LAYOUTS = """
DECODE = struct.Struct("@6q15qif2qPqPPq")
BEAM = struct.Struct("@8qi0q")
VIEW = struct.Struct("@P2q")
"""
_NO_GPU = "import ctypes, struct, sys" + LAYOUTS + r"""
sys.path.insert(0, ROOT)
import gated_delta_rule_50_gb300 as gdn
lib, P, I, C = gdn.load_library(), ctypes.c_void_p, ctypes.c_int64, ctypes.c_char_p
lib.gdn_recurrent.argtypes = lib.gdn_tree.argtypes = [C] + [P] * 9
lib.gdn_beam_search_workspace_bytes.argtypes = [C]
lib.gdn_beam_search_workspace_bytes.restype = ctypes.c_size_t
lib.gdn_beam_search.argtypes = [C] + [P] * 8 + [ctypes.c_size_t, P]
lib.gdn_reorder_states.argtypes = [C] + [I] * 4 + [P] * 3
A = 4096
def prob(B=2, T=3, Hq=2, Hv=4, K=128, V=128, io_dtype=1, n_slots=5, slot_stride=4 * 128 * 128, state_indices=0, n_seqs=2,
         cu_seqlens=0, token_indices=0, n_steps=0):
    return DECODE.pack(B, T, Hq, Hv, K, V, *[128] * 15, io_dtype, 0.1, n_slots, slot_stride, state_indices, n_seqs,
                          cu_seqlens, token_indices, n_steps)
def rec(p, q=A, k=A, v=A, g=A, b=A, s=A, out=None, o=A):
    return lib.gdn_recurrent(p, q, k, v, g, b, s, out, o, None)
def tree(p, q=A, k=A, v=A, g=A, b=A, par=A, s=A, o=A):
    return lib.gdn_tree(p, q, k, v, g, b, par, s, o, None)
out = dict(
    null=lib.gdn_recurrent(None, *[A] * 8, None),
    k=rec(prob(), k=None), state=rec(prob(), s=None), q_only=rec(prob(), o=None), o_only=rec(prob(), q=None),
    q_odd=rec(prob(), q=A + 1), state_odd=rec(prob(), s=A + 8), stride=rec(prob(slot_stride=4 * 128 * 128 + 2)),
    small=rec(prob(slot_stride=128)), slots=rec(prob(n_slots=1)), heads=rec(prob(Hv=3)), width=rec(prob(K=96)),
    dtype=rec(prob(io_dtype=3)), negative=rec(prob(T=-1)), seqs=rec(prob(n_seqs=1)),
    cu_batch=rec(prob(cu_seqlens=A)), cu_list=rec(prob(B=1, n_seqs=1, cu_seqlens=A, token_indices=A)),
    overlap=rec(prob(), out=A + 4 * 128 * 128 * 4 * 4), nothing=rec(prob(B=0, n_seqs=0)),
    t_parents=tree(prob(), par=None), t_wide=tree(prob(T=65)), t_cu=tree(prob(B=1, n_seqs=1, cu_seqlens=A)),
    t_nothing=tree(prob(T=0)))
def beam(B=2, W=3, vocab=100, n=4, logits_dtype=1):
    return BEAM.pack(B, W, vocab, n, 300, 100, 0, 0, logits_dtype)
def search(p, logits=A, scores=A, o=A, ws=A, n=1 << 30):
    return lib.gdn_beam_search(p, logits, scores, None, None, o, A, A, ws, n, None)
out.update(b_ws=lib.gdn_beam_search_workspace_bytes(beam()) > 0, b_bad=lib.gdn_beam_search_workspace_bytes(beam(n=0)),
    b_n=search(beam(n=65)), b_W=search(beam(W=65)), b_vocab=search(beam(vocab=(1 << 20) + 1)), b_zero=search(beam(vocab=0)),
    b_dtype=search(beam(logits_dtype=5)), b_null=search(beam(), logits=None), b_odd=search(beam(), logits=A + 1),
    b_small=search(beam(), n=64), b_ws_odd=search(beam(), ws=A + 16), b_nothing=search(beam(B=0)))
def reorder(data=A, stride=64, size=64, slots=8, B=2, W=4, par=A):
    return lib.gdn_reorder_states(VIEW.pack(data or 0, stride, size), 1, slots, B, W, par, None, None)
out.update(r_null=reorder(data=None), r_stride=reorder(stride=32), r_slots=reorder(slots=7), r_W=reorder(W=65),
    r_parents=reorder(par=None), r_nothing=reorder(B=0), r_views=lib.gdn_reorder_states(None, 1, 8, 2, 4, A, None, None))
print(repr(out))
"""


def test_c_entries_refuse_on_the_host():
    import ast
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + _NO_GPU], env=dict(os.environ, CUDA_VISIBLE_DEVICES=""),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    got = ast.literal_eval(r.stdout.strip().splitlines()[-1])
    invalid = ["null", "k", "state", "q_only", "o_only", "q_odd", "state_odd", "stride", "small", "slots", "heads", "dtype",
               "negative", "seqs", "cu_batch", "cu_list", "overlap", "t_parents", "t_cu", "b_zero", "b_dtype", "b_null",
               "b_odd", "r_null", "r_stride", "r_slots", "r_parents", "r_views"]
    want = {**{n: 1 for n in invalid}, **{n: 2 for n in ("width", "t_wide", "b_n", "b_W", "b_vocab", "r_W")},
            **{n: 3 for n in ("b_small", "b_ws_odd")}, **{n: 0 for n in ("nothing", "t_nothing", "b_nothing", "r_nothing", "b_bad")},
            "b_ws": True}
    assert got == want


def test_struct_sizes_match_the_header(tmp_path):
    """The layouts that the test above packs have the C structures' sizes."""
    import shutil
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "gdn.h"\nint main(void){printf("%zu %zu %zu\\n", sizeof(gdn_decode_problem), '
                   'sizeof(gdn_beam_problem), sizeof(gdn_state_view));return 0;}\n')
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(n) for n in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    layouts = {"struct": struct}
    exec(LAYOUTS, layouts)
    assert sizes == [layouts[n].size for n in ("DECODE", "BEAM", "VIEW")]

"""The largest numbers of rows and tokens of gdn_sample, in a process that sees no GPU: what is refused is not launched."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_PROGRAM = r"""
import ctypes as C, re
import gated_delta_rule_50_gb300 as gdn
lib = gdn.load_library()
text = open("include/gdn.h").read()
rows, vocab = (1 << int(re.search(r"#define GDN_SAMPLE_%s_MAX \(1 << (\d+)\)" % n, text).group(1)) for n in ("ROWS", "VOCAB"))
class Q(C.Structure): _fields_ = ([(n, C.c_int64) for n in ("B", "vocab", "logits_row", "mask_row")] + [("dtype", C.c_int)] +
                                  [(n, C.c_void_p) for n in ("temperatures", "top_ps", "min_ps", "top_ks")] +
                                  [(n, C.c_float) for n in ("temperature", "top_p", "min_p")] + [("top_k", C.c_int32)])
x = C.c_void_p(4096)
def sample(B, vocab, logits=x):
    return lib.gdn_sample(C.byref(Q(B, vocab, vocab, 0, 1)), logits, x, None, x, x, None)
assert sample(rows + 1, 10) == 2 and sample(1, vocab + 1) == 2
assert sample(rows, vocab, None) == 1 and sample(rows, 10, None) == 1  # in range: refused for what is missing
print("as expected")
"""


def test_limits():
    r = subprocess.run([sys.executable, "-c", _PROGRAM], capture_output=True, text=True, cwd=ROOT,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT))
    assert r.returncode == 0 and "as expected" in r.stdout, r.stdout + r.stderr

"""Where the segments of a sequence begin and end, for sequences of up to 2^31 - 65 tokens: tests/c/linear_parts.cu calls the
kernels' own function on the host (their outputs would fill the GPU's memory)."""
import os
import subprocess

from gated_delta_rule_50_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_segments_follow_each_other(tmp_path):
    exe = str(tmp_path / "linear_parts")
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, os.path.join(ROOT, "tests", "c", "linear_parts.cu"),
                    "-o", exe], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout

"""Builds libgdn.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc, and
beside it, where it is asked for, the extension module that the decoding calls of
the Python package go through (g++, against PyTorch's and Python's headers).

Each translation unit under csrc/ is compiled in parallel, then linked into
``gated_delta_rule_50_gb300/_build/libgdn.so``; that needs nvcc alone.
csrc/binding.cpp becomes ``_build/_gdn_decode.so``, which links to it.  Each has a
stamp that skips the rebuild when nothing changed: sources and flags, and for the
extension module the versions of PyTorch and Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libgdn.so")
BINDING = os.path.join(BUILD, "_gdn_decode.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch() -> str:
    """PyTorch's folder, found without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch not found")
    return list(spec.submodule_search_locations)[0]


def _digest(files, *texts) -> str:
    h = hashlib.sha256()
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    for t in texts:
        h.update(t.encode())
    return h.hexdigest()


def _stamp(extra) -> str:
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return _digest(sorted(_sources() + headers), " ".join(ARCH + NVCC_FLAGS + list(extra)))


def _binding_stamp() -> str:
    files = [os.path.join(CSRC, "binding.cpp"), *sorted(glob.glob(os.path.join(INCLUDE, "*.h"))), os.path.join(_torch(), "version.py")]
    return _digest(files, sys.version)


def _stamped(name, stamp) -> bool:
    path = os.path.join(BUILD, name)
    if not os.path.exists(path):
        return False
    with open(path) as fh:
        return fh.read() == stamp


def _set_stamp(name, stamp) -> None:
    with open(os.path.join(BUILD, name), "w") as fh:
        fh.write(stamp)


def _run(cmd, what) -> subprocess.CompletedProcess:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r


def build(verbose: bool = False, extra_flags=(), force: bool = False) -> str:
    """libgdn.so; its path."""
    os.makedirs(BUILD, exist_ok=True)
    stamp = _stamp(extra_flags)
    if not force and os.path.exists(LIB) and _stamped("stamp", stamp):
        return LIB
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        r = _run([nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj], f"nvcc failed on {src}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], "link failed")
    os.replace(tmp, LIB)
    _set_stamp("stamp", stamp)
    return LIB


def _compile_binding() -> str:
    if shutil.which("g++") is None:
        raise RuntimeError("g++ not found: the decoding calls' extension module needs it")
    torch, obj = _torch(), os.path.join(BUILD, "binding.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-w", *[x for i in include for x in ("-I", i)], "-c",
          os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ failed on binding.cpp")
    return obj


def build_binding(verbose: bool = False) -> str:
    """The extension module, and the library that it links to; the module's path."""
    os.makedirs(BUILD, exist_ok=True)
    stamp = _binding_stamp()
    if os.path.exists(BINDING) and _stamped("binding_stamp", stamp):
        build(verbose)
        return BINDING
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # beside nvcc
        obj = ex.submit(_compile_binding)
        build(verbose)
        obj = obj.result()
    torch_lib = os.path.join(_torch(), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-lgdn", "-L", torch_lib, "-ltorch_python", "-ltorch_cuda",
          "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"], "link of the binding failed")
    os.replace(tmp, BINDING)
    _set_stamp("binding_stamp", stamp)
    return BINDING


if __name__ == "__main__":
    print(build(verbose=True, force=True))

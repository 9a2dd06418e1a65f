"""What each of the two built files needs: the library of the C interface nvcc alone, the extension module of the
decoding calls the host compiler, PyTorch and this Python besides."""
import os
import stat
import sys

import pytest

import gated_delta_rule_50_gb300.build as b


@pytest.fixture
def empty(tmp_path, monkeypatch):
    """A build folder of its own and compilers that only write their output file, and a line of what they were asked."""
    log = tmp_path / "calls"
    tool = tmp_path / "bin" / "tool"
    tool.parent.mkdir()
    tool.write_text(f"#!{sys.executable}\nimport sys\nopen({str(log)!r}, 'a').write(' '.join(sys.argv) + '\\n')\n"
                    "open(sys.argv[sys.argv.index('-o') + 1], 'w').write('built')\n")
    tool.chmod(tool.stat().st_mode | stat.S_IXUSR)
    os.symlink(tool, tool.parent / "nvcc")
    monkeypatch.setenv("NVCC", str(tool.parent / "nvcc"))
    monkeypatch.setenv("PATH", str(tool.parent))
    out = tmp_path / "out"
    monkeypatch.setattr(b, "BUILD", str(out))
    monkeypatch.setattr(b, "LIB", str(out / "libgdn.so"))
    monkeypatch.setattr(b, "BINDING", str(out / "_gdn_decode.so"))

    def calls():
        text = log.read_text() if log.exists() else ""
        log.write_text("")
        return text.splitlines()
    return tool.parent, calls


def test_library_needs_nvcc_alone(empty, monkeypatch):
    _, calls = empty

    def gone():
        raise RuntimeError("PyTorch not found")
    monkeypatch.setattr(b, "_torch", gone)
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert len(calls()) == len(b._sources()) + 1
    assert b.build() == b.LIB and calls() == []
    with pytest.raises(RuntimeError, match="PyTorch"):
        b.build_binding()


def test_binding_says_what_is_missing(empty):
    with pytest.raises((RuntimeError, OSError), match=r"g\+\+"):
        b.build_binding()


def test_binding_is_built_for_this_python_and_pytorch(empty, monkeypatch, tmp_path):
    tools, calls = empty
    os.symlink(tools / "tool", tools / "g++")
    assert b.build_binding() == b.BINDING and os.path.exists(b.BINDING) and os.path.exists(b.LIB)
    calls()
    assert b.build_binding() == b.BINDING and calls() == []
    monkeypatch.setattr(sys, "version", sys.version + " another")
    b.build_binding()
    names = calls()
    assert names and all("nvcc" not in n.split()[0] for n in names)  # the library stays as it is
    torch = tmp_path / "torch"
    (torch / "include").mkdir(parents=True)
    (torch / "version.py").write_text("another")
    monkeypatch.setattr(b, "_torch", lambda: str(torch))
    b.build_binding()
    names = calls()
    assert names and all("nvcc" not in n.split()[0] for n in names)

"""libtwell is built from hipcc alone; the Python module beside it needs torch's
headers on top, and a failure there leaves the library built."""
import os
import subprocess

import pytest

from activation_sparse_feedforward_gate_amd import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build of one small source in a folder of its own, with host compilers
    of other names than hipcc out of reach."""
    src, out = tmp_path / "csrc", tmp_path / "lib"
    src.mkdir()
    (src / "one.cpp").write_text('extern "C" int twell_one() { return 1; }\n')
    for name, value in (("CSRC", src), ("BUILD", tmp_path / "obj"), ("LIBDIR", out), ("LIB", out / "libtwell.so"),
                        ("BIND", out / "_twell_bind.so")):
        monkeypatch.setattr(B, name, str(value))
    monkeypatch.setattr(B, "SOURCES", ["one.cpp"])
    real = subprocess.run

    def run(cmd, *a, **k):
        assert os.path.basename(cmd[0]) == os.path.basename(B.HIPCC), cmd[0]
        return real(cmd, *a, **k)
    monkeypatch.setattr(subprocess, "run", run)
    return out


def test_a_module_that_does_not_compile_leaves_the_library(tree):
    with open(os.path.join(B.CSRC, "bind.cpp"), "w") as f:
        f.write("#error no module\n")
    with pytest.raises(RuntimeError, match="bind.cpp"):
        B.build(jobs=1, verbose=False)
    assert (tree / "libtwell.so").exists() and not (tree / "_twell_bind.so").exists()


def test_without_torch_the_library_is_built(tree, monkeypatch, capsys):
    import builtins
    real = builtins.__import__

    def no_torch(name, *a, **k):
        if name.split(".")[0] == "torch":
            raise ImportError(name)
        return real(name, *a, **k)
    monkeypatch.setattr(builtins, "__import__", no_torch)
    B.build(jobs=1)
    assert (tree / "libtwell.so").exists() and not (tree / "_twell_bind.so").exists()
    assert "torch" in capsys.readouterr().out

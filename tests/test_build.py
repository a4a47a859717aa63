"""What the build makes anew, with compilers that only write files in their place."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_313_gb300 import build as B


class Compilers:
    """Stands in for subprocess.run: each command writes its output file; `broken` names outputs that fail."""

    def __init__(self):
        self.made, self.broken = [], set()

    def __call__(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".tmp")[0]
        if name in self.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "broken")
        with open(out, "w") as f:
            f.write(name)
        self.made.append(name)
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package of its own: sources, a PyTorch of a version, and compilers."""
    csrc, inc, torch, out = (tmp_path / n for n in ("csrc", "include", "torch", "_build"))
    for d in (csrc, inc, torch):
        d.mkdir()
    for f in (csrc / "a.cu", csrc / "b.cu", csrc / "c.cuh", csrc / "bind.cpp", inc / "pa.h"):
        f.write_text("")
    (torch / "__init__.py").write_text("")
    (torch / "version.py").write_text("__version__ = '1'")
    for name, value in (("CSRC", csrc), ("INCLUDE", inc), ("BUILD", out), ("LIB", out / "libpa.so"),
                        ("BIND", out / "_pa_bind.so")):
        monkeypatch.setattr(B, name, str(value))
    monkeypatch.setattr(B, "_torch_dir", lambda: str(torch))
    monkeypatch.setattr(B, "nvcc", lambda: sys.executable)
    cc = Compilers()
    monkeypatch.setattr(B.subprocess, "run", cc)
    cc.torch, cc.csrc = torch, csrc
    return cc


def _newer(path):
    t = max(os.path.getmtime(f) for f in (B.LIB, B.BIND)) + 10
    os.utime(path, (t, t))


def _made(cc):
    made, cc.made = sorted(cc.made), []
    return made


ALL = ["_pa_bind.so", "a.o", "b.o", "bind.o", "libpa.so"]


def test_builds_both_once(tree):
    assert B.build() == B.LIB and _made(tree) == ALL
    B.build()
    assert _made(tree) == []
    B.build(force=True)
    assert _made(tree) == ALL


def test_a_binding_that_failed_to_link_is_not_kept(tree):
    """After the library was replaced, an older binding would call it with the signatures of before."""
    B.build()
    _made(tree)
    for f in ("a.cu", "bind.cpp"):
        _newer(tree.csrc / f)
    tree.broken = {"_pa_bind.so"}
    with pytest.raises(RuntimeError, match="binding"):
        B.build()
    os.utime(B.LIB, (os.path.getmtime(tree.csrc / "a.cu") + 1,) * 2)  # (the library was made after its sources)
    _made(tree)
    tree.broken = set()
    B.build()
    assert "_pa_bind.so" in _made(tree)


def test_a_binding_of_another_pytorch_is_made_anew(tree):
    B.build()
    _made(tree)
    (tree.torch / "version.py").write_text("__version__ = '2'")
    t = os.path.getmtime(B.BIND) - 100  # (an installed file is older)
    os.utime(tree.torch / "version.py", (t, t))
    B.build()
    assert _made(tree) == ["_pa_bind.so", "bind.o"]
    B.build()
    assert _made(tree) == []


@pytest.mark.parametrize("broken", ["bind.o", "_pa_bind.so"])
def test_the_library_is_linked_where_the_binding_fails(tree, broken):
    tree.broken = {broken}
    with pytest.raises(RuntimeError):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BIND)


def test_the_library_needs_no_pytorch(tree, monkeypatch):
    monkeypatch.setattr(B, "_torch_dir", lambda: None)
    assert B.build() == B.LIB and _made(tree) == ["a.o", "b.o", "libpa.so"]
    B.build()
    assert _made(tree) == []

"""build() fails where a compiler does, and then leaves both libraries as they were (no GPU)."""
import os
import stat

import pytest

from direct_implicit_gemm_amd import build as B


def compiler(path, works):
    """A program that writes its -o argument, or fails."""
    path.write_text("#!/bin/sh\n" + ("" if works else "echo 'no such type' >&2; exit 1\n") +
                    'while [ $# -gt 0 ]; do\n  if [ "$1" = -o ]; then echo new > "$2"; fi\n'
                    "  shift\ndone\n")
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Both libraries built before, and a build() that writes beside them."""
    for name, at in (("LIB_PATH", "libconv.so"), ("CALLS_PATH", "_torch_calls.so")):
        (tmp_path / at).write_text("old\n")
        monkeypatch.setattr(B, name, str(tmp_path / at))
    return tmp_path


def state(tree):
    return sorted(f for f in os.listdir(tree) if ".so" in f), \
        [(tree / f).read_text().strip() for f in ("libconv.so", "_torch_calls.so")]


FILES = ["_torch_calls.so", "libconv.so"]


def test_both_are_replaced(tree, monkeypatch):
    monkeypatch.setattr(B, "HIPCC", compiler(tree / "hipcc", True))
    monkeypatch.setattr(B, "CXX", compiler(tree / "g++", True))
    assert B.build(verbose=False) == str(tree / "libconv.so")
    assert state(tree) == (FILES, ["new", "new"])


@pytest.mark.parametrize("hipcc,cxx", [(True, False), (False, True), (False, False)])
def test_a_failing_compiler_fails_the_build(tree, monkeypatch, hipcc, cxx):
    monkeypatch.setattr(B, "HIPCC", compiler(tree / "hipcc", hipcc))
    monkeypatch.setattr(B, "CXX", compiler(tree / "g++", cxx))
    with pytest.raises(RuntimeError, match="no such type"):
        B.build(verbose=False)
    assert state(tree) == (FILES, ["old", "old"])


def test_a_missing_torch_fails_the_build(tree, monkeypatch):
    import importlib.util
    found = importlib.util.find_spec
    monkeypatch.setattr(B, "HIPCC", compiler(tree / "hipcc", True))
    monkeypatch.setattr(B, "CXX", compiler(tree / "g++", True))
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else found(name, *a))
    with pytest.raises(RuntimeError, match="torch is not installed"):
        B.build(verbose=False)
    assert state(tree) == (FILES, ["old", "old"])

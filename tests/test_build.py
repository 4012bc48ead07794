"""The build: the C library does not depend on what only the calls on tensors
need (torch's and Python's headers).  The compilers are stood in for."""

import os

import pytest

from block_quantized_expert_amd import build as build_mod


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build() into tmp_path with commands that only create their output;
    returns the list of (source or output) that were asked for."""
    monkeypatch.setattr(build_mod, "BUILD_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(build_mod, "LIB", str(tmp_path / "lib" / "libmoe.so"))
    monkeypatch.setattr(build_mod, "CALLS", str(tmp_path / "lib" / "tensor_calls.so"))
    monkeypatch.setattr(build_mod, "_torch_flags", lambda: [])
    monkeypatch.setattr(build_mod, "_torch_libs", lambda: [])
    asked, fail = [], []

    def run(cmd):
        out = cmd[cmd.index("-o") + 1]
        asked.append(os.path.basename(out))
        if any(f in out for f in fail):
            raise RuntimeError("command failed: " + out)
        with open(out, "w") as f:
            f.write("new")
        return ""

    monkeypatch.setattr(build_mod, "_run", run)
    return tmp_path, asked, fail


def _read(path):
    return path.read_text() if path.exists() else None


def test_builds_both(tree):
    path, asked, _ = tree
    assert build_mod.build() == str(path / "lib" / "libmoe.so")
    assert _read(path / "lib" / "libmoe.so") == _read(path / "lib" / "tensor_calls.so") == "new"
    assert len(asked) == len(build_mod.HIP_SOURCES) + len(build_mod.HOST_SOURCES) + 3


def test_library_is_there_when_the_calls_on_tensors_fail(tree):
    path, _, fail = tree
    fail.append("tensor_calls")
    with pytest.raises(RuntimeError, match="tensor_calls"):
        build_mod.build()
    assert _read(path / "lib" / "libmoe.so") == "new"


def test_library_is_built_without_torch(tree, monkeypatch, capsys):
    path, asked, _ = tree

    def none():
        raise ImportError("No module named 'torch'")

    monkeypatch.setattr(build_mod, "_torch_flags", none)
    (path / "lib").mkdir()
    (path / "lib" / "tensor_calls.so").write_text("of an older library")
    build_mod.build()
    assert _read(path / "lib" / "libmoe.so") == "new"
    assert _read(path / "lib" / "tensor_calls.so") is None
    assert not any("tensor_calls" in a for a in asked)
    assert "tensor_calls.so is not built" in capsys.readouterr().err


def test_a_failing_kernel_fails_the_build(tree):
    path, _, fail = tree
    fail.append("moe_rows")
    with pytest.raises(RuntimeError, match="moe_rows"):
        build_mod.build()
    assert _read(path / "lib" / "libmoe.so") is None

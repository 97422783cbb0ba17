"""What the build and the binding do without torch's headers, a C++ compiler or the
CPython module (no GPU needed; nothing is compiled here)."""

from __future__ import annotations

import builtins
import os
import shutil
import subprocess
import sys
import types

import pytest
import torch

import swiglu_activation_amd as sw
from swiglu_activation_amd import build


@pytest.fixture
def stale(tmp_path, monkeypatch):
    """A module of an earlier build in the place of this one's."""
    p = tmp_path / "_torch_calls.so"
    p.write_bytes(b"old")
    monkeypatch.setattr(build, "CALLS", str(p))
    return p


def test_no_compiler(stale, monkeypatch, capsys):
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert build.build_calls() is None
    assert not stale.exists() and "no C++ compiler" in capsys.readouterr().err


def test_no_torch(stale, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build_calls() is None
    assert not stale.exists() and "torch" in capsys.readouterr().err


def test_no_headers(stale, monkeypatch, tmp_path, capsys):
    monkeypatch.setitem(sys.modules, "torch", types.SimpleNamespace(__file__=str(tmp_path / "torch" / "__init__.py")))
    assert build.build_calls() is None
    assert not stale.exists() and "EmptyTensor.h" in capsys.readouterr().err


def test_the_library_and_the_client_come_first(stale, monkeypatch, tmp_path):
    """A module that does not compile is an error, and leaves a library and a client."""
    ran = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        ran.append(os.path.basename(out))
        failed = build.CALLS_SRC in cmd
        if not failed:
            open(out, "wb").close()
        return subprocess.CompletedProcess(cmd, int(failed), "", "no such thing")

    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "CLIENT", str(tmp_path / "client"))
    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="torch calls"):
        build.build()
    assert ran == ["lib.so.tmp", "client", "_torch_calls.so.tmp"]
    which = shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda name: None if name in ("g++", "c++") else which(name))
    ran.clear()
    assert build.build() == str(tmp_path / "lib.so") and ran == ["lib.so.tmp", "client"]


def test_calls_without_the_module_go_through_ctypes(monkeypatch):
    real = builtins.__import__

    def without(name, globals=None, locals=None, fromlist=(), level=0):
        if "_torch_calls" in (fromlist or ()):
            raise ImportError("no module for this test")
        return real(name, globals, locals, fromlist, level)

    monkeypatch.setattr(sw, "_calls", None)
    monkeypatch.setattr(builtins, "__import__", without)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        calls = sw._native()
    assert sw._native() is calls
    a, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 6, 8, dtype=torch.bfloat16)
    for name, n in (("mm", 3), ("fc1", 4), ("mm_dgrad", 3), ("mm_wgrad", 4), ("ckpt8_fwd", 2), ("ckpt8_bwd", 6)):
        assert getattr(calls, name)(*[a] * n) is None
    with pytest.raises(ValueError, match="HIP device"):      # the binding's own refusal of host tensors
        sw.swiglu_grouped_mm(a, w, torch.zeros(2, dtype=torch.int32))

"""The build of the Python module beside the library: what it links to, and
machines without torch, with a torch that has no CUDA, or without Python.h."""
import importlib.machinery
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest


def build_module():
    import __graft_entry__ as g
    return g._load_pkg_build()


SCRIPT = """
import os, sys
sys.path.insert(0, {root!r})
import int4_expert_ffn_router_b200 as coli
import torch
coli._ops()
loaded = {{l.split(None, 5)[5].strip() for l in open("/proc/self/maps") if "libcoli_moe.so" in l}}
assert loaded == {{os.path.realpath(os.path.join(coli.HERE, "libcoli_moe.so"))}}, loaded
assert coli.HERE.startswith({root!r}), coli.HERE
print("one library")
"""


def test_a_copied_tree_runs_its_own_library(tmp_path):
    """The module finds the library beside it, wherever the package lies, and no second one."""
    pytest.importorskip("torch")
    b = build_module()
    if not (os.path.exists(b.SO) and os.path.exists(b.BINDING_SO)):
        b.build()
    copy = tmp_path / "int4_expert_ffn_router_b200"
    copy.mkdir()
    for name in ("__init__.py", "build.py", "libcoli_moe.so", "_binding.so"):
        shutil.copy(os.path.join(b.HERE, name), copy / name)
    p = subprocess.run([sys.executable, "-c", SCRIPT.format(root=str(tmp_path))], cwd=tmp_path, capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0 and "one library" in p.stdout, p.stderr[-2000:]


def test_build_without_torch(monkeypatch, capsys):
    """The C library and its ctypes layer need no torch: the build goes on without the module."""
    b = build_module()
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, package=None: None)
    monkeypatch.setattr(subprocess, "check_call", lambda *a, **k: pytest.fail("nothing to compile"))
    assert b.build_binding() is None
    assert "torch" in capsys.readouterr().out


def test_build_with_a_torch_without_cuda(monkeypatch, capsys, tmp_path):
    b = build_module()
    (tmp_path / "lib").mkdir()
    spec = importlib.machinery.ModuleSpec("torch", None, origin=str(tmp_path / "__init__.py"))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, package=None: spec)
    monkeypatch.setattr(subprocess, "check_call", lambda *a, **k: pytest.fail("nothing to link to"))
    assert b.build_binding() is None
    assert "CUDA" in capsys.readouterr().out


def test_build_without_python_headers(monkeypatch, capsys, tmp_path):
    import sysconfig
    pytest.importorskip("torch")
    b = build_module()
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    monkeypatch.setattr(subprocess, "check_call", lambda *a, **k: pytest.fail("nothing to compile against"))
    assert b.build_binding() is None
    assert "Python.h" in capsys.readouterr().out

"""When the native part of the binding is built again, and what its absence leaves (CPU)."""
import os
import sysconfig

import pytest
import torch

from fp8_fp4_moe_b200 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_a_fresh_build_is_kept():
    t = os.path.getmtime(build.OPS)
    assert build.build_ops() == build.OPS and os.path.getmtime(build.OPS) == t


def test_another_torch_or_interpreter_makes_it_stale(monkeypatch):
    assert not build.ops_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.99.0")
        assert build.ops_stale()
    with monkeypatch.context() as m:
        m.setattr(build.sys, "version", "3.99.0")
        assert build.ops_stale()
    with monkeypatch.context() as m:
        m.setattr(build, "OPS_STAMP", build.OPS_STAMP + ".none")
        assert build.ops_stale()
    assert not build.ops_stale()


@pytest.mark.parametrize("what", ["Python.h", "g++"])
def test_the_library_builds_without_what_the_native_binding_needs(monkeypatch, tmp_path, what):
    monkeypatch.setattr(build, "OPS", str(tmp_path / "_moe_ops.so"))
    if what == "g++":
        which = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" else which(name))
    else:
        path = sysconfig.get_path
        monkeypatch.setattr(sysconfig, "get_path", lambda name: str(tmp_path) if name == "include" else path(name))
    with pytest.warns(UserWarning, match="not built"):
        assert build.build() == build.LIB
    assert not os.path.exists(build.OPS)
    monkeypatch.undo()
    assert os.path.exists(build.OPS) and not build.ops_stale()

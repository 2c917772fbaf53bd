"""When the native part of the binding is built again (CPU)."""
import os

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

"""What the build takes as current, and what it leaves when a part of it fails.  Nothing is compiled here: the compilers
are stand-ins that write the file they are asked for."""
import os
import subprocess
import types

import pytest

import quantized_routed_expert_router_gb300 as moe
from quantized_routed_expert_router_gb300 import _build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """a build into tmp_path; the commands that were run, and the programs that fail"""
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(_build, "SO", str(tmp_path / "_moe.so"))
    monkeypatch.setattr(_build, "CALLS_SO", str(tmp_path / "_calls.so"))
    at = types.SimpleNamespace(ran=[], fails=())

    def run(cmd, **_):
        name = os.path.basename(cmd[0])
        at.ran.append(name)
        if name in at.fails:
            return types.SimpleNamespace(returncode=1, stdout="", stderr=f"{name}: no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(name)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(subprocess, "run", run)
    return at


def test_a_second_build_does_nothing(elsewhere):
    assert _build.build() == _build.SO and os.path.exists(_build.CALLS_SO) and _build.up_to_date()
    elsewhere.ran.clear()
    _build.build()
    assert not elsewhere.ran


def test_the_library_is_there_when_the_binding_fails(elsewhere):
    elsewhere.fails = ("g++",)
    with pytest.raises(RuntimeError, match="no such header"):
        _build.build()
    assert os.path.exists(_build.SO) and not os.path.exists(_build.CALLS_SO)
    assert _build.lib_up_to_date() and not _build.up_to_date()
    # only the binding is left to build
    elsewhere.fails = ()
    elsewhere.ran.clear()
    _build.build()
    assert set(elsewhere.ran) == {"g++"} and _build.up_to_date()


def test_a_binding_for_another_torch_is_not_current(elsewhere, monkeypatch):
    import torch
    _build.build()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert _build.lib_up_to_date() and not _build.calls_up_to_date() and not _build.up_to_date()
    elsewhere.ran.clear()
    _build.build()
    assert set(elsewhere.ran) == {"g++"} and _build.up_to_date()


def test_a_binding_for_another_torch_is_not_used(monkeypatch):
    import torch
    monkeypatch.setattr(moe, "_bound", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    with pytest.raises(RuntimeError, match="0.0.0"):
        moe.moe_expert_order(None, 4)

"""When the operators' compiled binding is built again."""
from __future__ import annotations

import importlib.util
import pathlib

import pytest

import moe_grouped_gemm_08_b200 as fg


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module with its outputs under tmp_path and its compiler replaced by one that writes a file."""
    spec = importlib.util.spec_from_file_location("_build_of_the_test", pathlib.Path(fg.__file__).parent / "build.py")
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.GEN, module.BINDING, module.runs = tmp_path / "gen", tmp_path / "_operators.so", []

    def compiler(cmd):
        module.runs.append(cmd)
        pathlib.Path(cmd[cmd.index("-o") + 1]).write_bytes(b"")

    monkeypatch.setattr(module.subprocess, "check_call", compiler)
    return module


def test_binding_is_built_again_for_another_torch(build, monkeypatch):
    build.build_binding()
    build.build_binding()
    assert len(build.runs) == 1  # nothing changed
    monkeypatch.setattr(build, "torch_version", lambda: "99.0")
    build.build_binding()
    assert len(build.runs) == 2
    build.build_binding()
    assert len(build.runs) == 2
    build.build_binding(force=True)
    assert len(build.runs) == 3

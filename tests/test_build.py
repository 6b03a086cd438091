"""The build's order and what it rebuilds, with stand-ins for the compilers (no
GPU, nothing is compiled)."""
import importlib
import os
import subprocess

import pytest

import fp8_routed_expert_gb300 as moe
from fp8_routed_expert_gb300 import _lib

build = importlib.import_module("fp8_routed_expert_gb300.build")


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """Compilers that note their output files, and make them unless told to fail."""
    class Tools:
        made, fail = [], ()

        def run(self, cmd, **kw):
            tool, out = os.path.basename(cmd[0]), cmd[cmd.index("-o") + 1]
            self.made.append((tool, os.path.basename(out).split(".tmp")[0]))
            if tool not in self.fail:
                open(out, "w").close()
            return subprocess.CompletedProcess(cmd, int(tool in self.fail), "", "")

    t = Tools()
    t.made, t.lib = [], str(tmp_path / "libfp8moe.so")
    monkeypatch.setattr(build, "LIB", t.lib)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/bin/nvcc")
    monkeypatch.setattr(build.subprocess, "run", t.run)
    monkeypatch.setattr(_lib, "PKG", str(tmp_path))
    return t


def test_the_library_needs_no_host_compiler(tools):
    tools.fail = ("g++",)
    with pytest.raises(RuntimeError, match="is built.*binding is not"):
        build.build()
    assert os.path.exists(tools.lib) and not os.path.exists(_lib.binding_path())
    # later, with one: the binding alone is made
    tools.made.clear()
    tools.fail = ()
    assert build.build() == tools.lib
    assert {tool for tool, _ in tools.made} == {"g++"} and os.path.exists(_lib.binding_path())
    tools.made.clear()
    build.build()
    assert tools.made == []
    build.build(force=True)
    assert ("nvcc", "libfp8moe.so") in tools.made and ("g++", os.path.basename(_lib.binding_path())) in tools.made


def test_another_torch_gets_a_binding_of_its_own(tools, monkeypatch):
    import torch
    build.build()
    first = _lib.binding_path()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    other = _lib.binding_path()
    assert other != first and not os.path.exists(other)
    monkeypatch.setattr(_lib, "_binding", None)
    with pytest.raises(RuntimeError, match="is not built"):
        moe._lib.torch_binding()
    tools.made.clear()
    build.build()
    assert os.path.exists(other) and os.path.exists(first) and {tool for tool, _ in tools.made} == {"g++"}


def test_a_failed_library_is_an_error(tools):
    tools.fail = ("nvcc",)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()
    assert not os.path.exists(tools.lib)

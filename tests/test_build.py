"""What the build of the library and of its binding asks for, on the CPU, with the compilers replaced by a record
of their commands."""
import os
import subprocess
import types

import pytest
import torch

from linear_attention_serving_02_gb300 import build


@pytest.fixture
def calls(monkeypatch, tmp_path):
    """Commands that the build runs; each makes its output file, or fails if its program is in calls.broken."""
    made = types.SimpleNamespace(commands=[], broken=())

    def run(cmd, **_):
        made.commands.append(cmd)
        name = os.path.basename(cmd[0])
        if name in made.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "no such thing")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libkda_gb300.so"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return made


def test_the_library_needs_neither_torch_nor_a_host_compiler(calls, monkeypatch):
    monkeypatch.setattr(build, "_torch_dir", lambda: pytest.fail("the library asked for torch"))
    calls.broken = ("g++",)
    assert build.build() == build.LIB and os.path.exists(build.LIB) and build.up_to_date()
    assert {os.path.basename(c[0]) for c in calls.commands} == {"nvcc"}
    assert not any("torch" in a or a.endswith(".cpp") for c in calls.commands for a in c)
    done = len(calls.commands)
    build.build()
    assert len(calls.commands) == done


def test_a_binding_that_does_not_compile_leaves_the_library(calls):
    calls.broken = ("g++",)
    with pytest.raises(RuntimeError, match=r"g\+\+ failed on .*kda_binding.cpp"):
        build.build_binding()
    assert build.up_to_date() and not os.path.exists(build.binding_path())


def test_another_torch_or_python_builds_its_own_binding(calls, monkeypatch):
    first = build.build_binding()
    assert os.path.exists(first) and build.binding_up_to_date()
    done = len(calls.commands)
    assert build.build_binding() == first and len(calls.commands) == done
    monkeypatch.setattr(torch, "__version__", "99.1+other")
    assert not build.binding_up_to_date()
    second = build.build_binding()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert not build.binding_up_to_date()
    third = build.build_binding()
    assert len({first, second, third}) == 3 and all(os.path.exists(p) for p in (first, second, third))
    assert sum(os.path.basename(c[0]) == "nvcc" for c in calls.commands) == sum(
        os.path.basename(c[0]) == "nvcc" for c in calls.commands[:done])

"""What the build makes and when it makes it anew, with the compilers stood in
for (no compilation): the C library needs neither torch nor the module for it,
and the module belongs to the torch it was compiled against."""
import os
import subprocess
import sys

import pytest
import torch

from routing_dispatch_grouped_router_gb300 import build


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """Paths under tmp_path, and the list of the commands run."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        os.makedirs(os.path.dirname(out), exist_ok=True)
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path / "lib"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib" / "libmok.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "lib" / os.path.basename(build.BINDING)))
    monkeypatch.setattr(subprocess, "run", run)
    return ran


def of_module(ran):
    return [c for c in ran if any("block_binding" in a for a in c)]


def test_library_without_torch(commands, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # `import torch` raises ImportError
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert len(commands) > 1 and not of_module(commands) and not os.path.exists(build.BINDING)
    assert build.up_to_date()
    commands.clear()
    build.build()
    assert not commands
    monkeypatch.undo()


def test_module_is_made_once_torch_is_there(commands, monkeypatch):
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        build.build()
    assert not build.up_to_date()
    commands.clear()
    build.build()
    assert os.path.exists(build.BINDING) and commands == of_module(commands)
    assert build.up_to_date()


def test_module_belongs_to_its_torch(commands, monkeypatch):
    build.build()
    assert of_module(commands) and build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert not build.up_to_date()
    commands.clear()
    build.build()
    assert commands and commands == of_module(commands)  # the library stays
    assert build.up_to_date()


def test_sources_newer_than_what_was_built(commands):
    build.build()
    now = os.path.getmtime(build.BINDING_SRC)
    for target in (build.LIB, build.BINDING):
        os.utime(target, (now - 10, now - 10))
        assert not build.up_to_date()
        build.build()
        assert build.up_to_date()

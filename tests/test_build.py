"""What the build makes and when, with the compilers replaced by a record of their commands."""
import os
import sys

import pytest

from bit_rank_compensated_b200 import build


@pytest.fixture
def commands(tmp_path, monkeypatch):
    made = []

    def run(cmd, check):
        assert check
        made.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libsvdq.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    return made


def test_binding_is_made_again_for_another_torch(commands, monkeypatch):
    torch = pytest.importorskip("torch")
    for version in (torch.__version__, "99.0", "99.1"):
        monkeypatch.setattr(torch, "__version__", version)
        before = len(commands)
        assert build.build_binding() == build.BINDING
        assert len(commands) == before + 1 and build.BINDING in commands[-1]
        build.build_binding()
        assert len(commands) == before + 1
    build.build_binding(force=True)
    assert len(commands) == before + 2


def test_binding_is_made_again_after_its_source(commands):
    pytest.importorskip("torch")
    build.build_binding()
    old = os.path.getmtime(os.path.join(build.CSRC, "binding.cpp")) - 10
    os.utime(build.BINDING, (old, old))
    build.build_binding()
    assert len(commands) == 2


def test_library_without_torch(commands, monkeypatch, capsys):
    """The library is a C ABI that needs no torch; only its Python calls do."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert commands and not any("binding.cpp" in word for cmd in commands for word in cmd)
    assert "torch" in capsys.readouterr().err

"""What build.py makes, from what, and when again (no compiler runs here: subprocess.run is replaced)."""

import subprocess
import sys
import time

import pytest

from muon_newton_schulz_expert_gb300 import build as mkbuild


class Compilers:
    """Stands in for subprocess.run: writes what the command would, and keeps the commands."""
    def __init__(self, fails=()):
        self.commands, self.fails = [], fails

    def __call__(self, cmd, **kw):
        self.commands.append(cmd)
        if any(f in c for f in self.fails for c in cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "not today")
        time.sleep(0.02)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def of(self, source):
        return [c for c in self.commands if any(a.endswith(source) for a in c)]


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """All outputs under a directory of their own, and no real compiler."""
    for name in ("LIB", "LIB_CHECKED", "BINDING"):
        monkeypatch.setattr(mkbuild, name, str(tmp_path / getattr(mkbuild, name).rsplit("/", 1)[1]))
    monkeypatch.setattr(mkbuild, "OUT_DIR", str(tmp_path))
    run = Compilers()
    monkeypatch.setattr(mkbuild.subprocess, "run", run)
    return run


def made(tmp_path):
    return {p.name for p in tmp_path.iterdir() if p.suffix == ".so"}


def test_the_library_needs_no_pytorch(elsewhere, monkeypatch, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", None)   # an import of it raises, as where there is none
    assert mkbuild.build() == mkbuild.LIB
    assert made(tmp_path) == {"libmuon.so"}
    mkbuild.build_all()
    assert made(tmp_path) == {"libmuon.so", "libmuon_checked.so"}


def test_a_binding_that_does_not_compile_is_an_error_after_the_library(elsewhere, tmp_path):
    elsewhere.fails = ("binding.cpp",)
    with pytest.raises(RuntimeError, match="not today"):
        mkbuild.build()
    assert made(tmp_path) == {"libmuon.so"}


@pytest.mark.parametrize("force", [False, True])
def test_build_all_makes_each_thing_once(elsewhere, tmp_path, force):
    assert mkbuild.build_all(force=force) == [mkbuild.LIB, mkbuild.LIB_CHECKED]
    assert made(tmp_path) == {"libmuon.so", "libmuon_checked.so", "muon_ops.so"}
    assert len(elsewhere.of("binding.cpp")) == 1
    assert all(len(elsewhere.of(s)) == 2 for s in mkbuild.SOURCES)
    elsewhere.commands.clear()
    mkbuild.build_all()
    assert not elsewhere.commands


def test_the_binding_is_made_again_for_another_torch(elsewhere, monkeypatch):
    mkbuild.build()
    mkbuild.build()
    assert len(elsewhere.of("binding.cpp")) == 1
    monkeypatch.setattr(mkbuild.importlib.metadata, "version", lambda name: "99.0")
    mkbuild.build()
    mkbuild.build()
    assert len(elsewhere.of("binding.cpp")) == 2
    monkeypatch.setattr(mkbuild.sys, "version_info", (3, 99, 0))
    mkbuild.build()
    assert len(elsewhere.of("binding.cpp")) == 3 and len(elsewhere.of(mkbuild.SOURCES[0])) == 1

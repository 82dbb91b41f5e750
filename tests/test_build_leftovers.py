"""A build that fails, or is interrupted, leaves no temporary files and no compilers behind. No GPU, nothing is compiled: the
commands of the build are replaced."""
import os

import pytest

from resharding_tensor_parallelism_gb300 import _build


@pytest.fixture
def place(tmp_path, monkeypatch):
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "TABLE", str(tmp_path / "table.so"))
    monkeypatch.setattr(_build, "HOST_SOURCES", [])
    monkeypatch.setattr(_build, "CUDA_SOURCES", ["a.cu"])
    monkeypatch.setattr(_build, "_table_command", lambda target: ["sh", "-c", "echo built > " + target])
    return tmp_path


def _files(place):
    return sorted(p.name for p in place.iterdir() if p.is_file())


def test_a_compilation_that_fails(place, monkeypatch):
    monkeypatch.setattr(_build, "_nvcc", lambda: "false")
    with pytest.raises(RuntimeError):
        _build.build(force=True)
    assert _files(place) == []


def test_a_link_that_fails(place, monkeypatch):
    compiler = place / "compiler"
    compiler.write_text("#!/bin/sh\ncase \"$*\" in *-shared*) echo half > %s.tmp%d; exit 1;; esac\n" % (_build.LIB, os.getpid()))
    compiler.chmod(0o755)
    monkeypatch.setattr(_build, "_nvcc", lambda: str(compiler))
    with pytest.raises(Exception):
        _build.build(force=True)
    assert _files(place) == ["compiler"]


def test_an_interrupted_build(place, monkeypatch):
    started = []
    popen = _build.subprocess.Popen

    class Popen(popen):
        def __init__(self, *args, **kw):
            started.append(self)
            super().__init__(*args, **kw)

        def communicate(self, *args, **kw):
            raise KeyboardInterrupt

    monkeypatch.setattr(_build, "_nvcc", lambda: "sleep")
    monkeypatch.setattr(_build, "ARCH", ["60"])
    monkeypatch.setattr(_build, "_table_command", lambda target: ["sh", "-c", "echo built > %s; exec sleep 60" % target])
    monkeypatch.setattr(_build.subprocess, "Popen", Popen)
    with pytest.raises(KeyboardInterrupt):
        _build.build(force=True)
    assert len(started) == 2 and all(p.poll() is not None for p in started)
    assert _files(place) == []


def test_a_build_that_works(place, monkeypatch):
    compiler = place / "compiler"
    compiler.write_text("#!/bin/sh\nwhile [ $# -gt 0 ]; do [ \"$1\" = -o ] && echo built > \"$2\"; shift; done\n")
    compiler.chmod(0o755)
    monkeypatch.setattr(_build, "_nvcc", lambda: str(compiler))
    assert _build.build(force=True) == _build.LIB
    assert _files(place) == ["compiler", "lib.so", "table.so"]

"""The library is built by hipcc alone, with or without what the Python
binding's compiled marshalling needs."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

from fp4_block_scaled_quantizer_amd import build


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """Compilers that only write the file they are asked for; the names of
    those that ran."""
    ran = []

    def run(cmd, **kwargs):
        ran.append(os.path.basename(cmd[0]))
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "OUT", str(tmp_path / "libfp4q.so"))
    monkeypatch.setattr(build, "ROW_CALLS_OUT", str(tmp_path / "_row_calls.so"))
    return ran


def test_without_torch_the_library_is_built(compiled, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it fails
    assert build.build() == build.OUT
    assert os.path.exists(build.OUT) and not os.path.exists(build.ROW_CALLS_OUT)
    assert set(compiled) == {"hipcc"}


def test_without_a_host_compiler_the_library_is_built(compiled, monkeypatch):
    which = shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda n, *a: None if "+" in n else which(n, *a))
    with pytest.raises(RuntimeError, match="host C"):
        build.build()
    assert os.path.exists(build.OUT) and not os.path.exists(build.ROW_CALLS_OUT)


def test_the_marshallings_failure_is_told_after_the_library(compiled, monkeypatch):
    def fails(verbose):
        raise RuntimeError("Python.h: no such file")

    monkeypatch.setattr(build, "_row_calls", fails)
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build()
    assert os.path.exists(build.OUT)


def test_both_are_built(compiled):
    build.build()
    assert os.path.exists(build.OUT) and os.path.exists(build.ROW_CALLS_OUT)
    assert compiled.count("hipcc") == len(build.SOURCES) + 1


def test_the_library_alone(compiled):
    assert build.build_library() == build.OUT
    assert set(compiled) == {"hipcc"} and not os.path.exists(build.ROW_CALLS_OUT)

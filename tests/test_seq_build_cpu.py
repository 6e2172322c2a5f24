"""The C library builds with hipcc alone: the Python binding of the sequence operators, which needs torch's headers and a
C++ compiler, takes hipcc where there is no other, and is left out where there is no torch."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILD = os.path.join(ROOT, "dynamic_convolution_amd", "build.py")


@pytest.fixture
def build(tmp_path):
    spec = importlib.util.spec_from_file_location("build_under_test", BUILD)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.BIND_LIB = str(tmp_path / "_seqbind.so")
    return m


def test_without_torch(tmp_path):
    """In a process that cannot import torch, with the kernels' compile and link left out."""
    code = """
import importlib.util, os, sys
sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("build_under_test", %r)
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
m.BUILD = %r
m.LIB, m.PROBE_LIB, m.BIND_LIB = (os.path.join(m.BUILD, n) for n in ("libdwconv.so", "libdwprobe.so", "_seqbind.so"))
m._compile = lambda src: src + ".o"
class Done:
    returncode, stdout = 0, ""
def run(cmd, **_):
    open(cmd[cmd.index("-o") + 1], "w").close()
    return Done
m.subprocess.run = run
m.build(verbose=True)
print(sorted(os.listdir(m.BUILD)))
""" % (BUILD, str(tmp_path))
    r = subprocess.run([sys.executable, "-c", code], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    assert "['libdwconv.so', 'libdwprobe.so']" in r.stdout and "_seqbind.so left out" in r.stdout, r.stdout


@pytest.mark.parametrize("cxx,gxx,want", [("my-c++", "/usr/bin/g++", "my-c++"), (None, "/usr/bin/g++", "g++"), (None, None, "hipcc")])
def test_compiler(build, monkeypatch, cxx, gxx, want):
    monkeypatch.delenv("CXX", raising=False)
    if cxx:
        monkeypatch.setenv("CXX", cxx)
    monkeypatch.setattr(build.shutil, "which", lambda name: gxx)
    seen = []

    def run(cmd, **_):
        seen.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "")

    monkeypatch.setattr(build.subprocess, "run", run)
    assert build.build_bind() == build.BIND_LIB and os.path.exists(build.BIND_LIB)
    assert os.path.basename(seen[0][0]) == want

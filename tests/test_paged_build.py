"""How the paged calls are built: what the translation units share, and several processes that build at once."""
from __future__ import annotations

import os
import subprocess
import sys
import time
import warnings

import pytest
import torch

import decode_context_attention_dcp_b200 as dcp
from decode_context_attention_dcp_b200 import _build, paged


def test_each_type_reads_its_own_timeout_counter(tmp_path):
    """Every translation unit has a counter of its own, so the function that reads it must not be merged with its
    namesakes by the linker, as functions of external linkage are that the compiler does not inline."""
    src, obj = tmp_path / "reader.cu", tmp_path / "reader.o"
    src.write_text('#include "dcp_paged_attention.cuh"\n'
                   "cudaError_t reader(unsigned long long &n) { return dcp_host::attention_timeouts(n, 1); }\n")
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O0", "-std=c++17", "-Xcompiler", "-fPIC,-O0", "-I", _build.INCLUDE,
                    "-I", _build.CSRC, "-c", str(src), "-o", str(obj)], check=True, capture_output=True, text=True)
    symbols = subprocess.run(["nm", "-C", str(obj)], check=True, capture_output=True, text=True).stdout
    found = [line for line in symbols.splitlines() if "attention_timeouts(" in line]
    assert found, "the reader was inlined: the test says nothing"
    assert all(line.split()[1] == "t" for line in found), found


BUILDER = """
import os, sys, time
import decode_context_attention_dcp_b200 as dcp
from decode_context_attention_dcp_b200 import _build, paged
pkg, what, start = sys.argv[1], sys.argv[2], float(sys.argv[3])
_build.PKG, _build.LIBRARY = pkg, os.path.join(pkg, "lib.so")
_build.BINDING = os.path.join(pkg, "binding.so")
_build.sources = lambda: [os.path.join(pkg, "one.cu")]

def run(cmd):  # a compiler that takes a while
    with open(os.path.join(pkg, "log"), "a") as fh:
        fh.write("run\\n")
    time.sleep(0.3)
    with open(cmd[cmd.index("-o") + 1], "w") as fh:
        fh.write("built")

_build._run = run
time.sleep(max(0.0, start - time.time()))
getattr(_build, what)()
"""


@pytest.mark.parametrize("what,lib,steps", [("build", "lib.so", 2), ("build_binding", "binding.so", 1)])
def test_several_processes_build_once(tmp_path, what, lib, steps):
    """Ranks whose first calls come together: one builds, the others wait, none fails."""
    (tmp_path / "one.cu").write_text("")
    start = str(time.time() + 8)
    code = [sys.executable, "-c", BUILDER, str(tmp_path), what, start]
    ranks = [subprocess.Popen(code, cwd=_build.ROOT, stderr=subprocess.PIPE, text=True) for _ in range(4)]
    errors = [p.communicate(timeout=120)[1] for p in ranks]
    assert [p.returncode for p in ranks] == [0] * 4, errors
    assert (tmp_path / "log").read_text() == "run\n" * steps
    assert (tmp_path / lib).read_text() == "built"
    assert len((tmp_path / (lib + ".sha256")).read_text().strip()) == 64
    assert sorted(os.listdir(tmp_path)) == sorted(["log", "one.cu", lib, lib + ".sha256"])


def test_the_binding_is_rebuilt_for_other_flags(monkeypatch):
    before = _build.binding_digest()
    monkeypatch.setattr(_build, "BINDING_FLAGS", [*_build.BINDING_FLAGS, "-DOTHER"])
    assert _build.binding_digest() != before


@pytest.mark.parametrize("error", [RuntimeError("g++ failed"), FileNotFoundError("g++"), PermissionError("package"),
                                   ImportError("undefined symbol")])
def test_calls_do_without_a_binding_that_cannot_be_built(monkeypatch, error):
    """One warning, then the Python code makes the calls (or, as here, says what is wrong with one)."""
    def fail():
        raise error

    monkeypatch.setattr(paged, "_native", None)
    monkeypatch.setattr(_build, "build_binding", fail)
    q, k = torch.zeros(3, 8, 64), torch.zeros(4, 16, 2, 64)
    args = (q, k, k, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.warns(RuntimeWarning, match="binding"), pytest.raises(ValueError, match="CUDA"):
        dcp.paged_attention(*args)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="CUDA"):
            dcp.paged_attention(*args)

"""How the paged calls are built: what the translation units share, and several processes that build at once."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from decode_context_attention_dcp_b200 import _build


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

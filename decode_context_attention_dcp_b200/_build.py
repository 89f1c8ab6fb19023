"""Build of libdcpcombine.so, in-tree, for sm_100a, and of the paged calls' torch binding.

    python -m decode_context_attention_dcp_b200._build        # build if stale
    python -m decode_context_attention_dcp_b200._build --force

nvcc cross-compiles without a GPU.  The library links the CUDA runtime
statically, so it does not depend on which libcudart the host process loaded.
The binding (_paged_binding.so) is host code: g++ against the headers of the
Python and torch that import it.
"""
from __future__ import annotations

import argparse
import concurrent.futures
import contextlib
import fcntl
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(PKG, "csrc")
LIBRARY = os.path.join(PKG, "libdcpcombine.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMPILE_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2"]
LINK_FLAGS = ["-shared", "--cudart", "static"]
BINDING_SOURCE = os.path.join(PKG, "binding", "paged_binding.cpp")
BINDING = os.path.join(PKG, "_paged_binding.so")
BINDING_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden"]
BINDING_LIBS = ["-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda", "-ldl"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the DCP combine library needs the CUDA toolkit to build")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def inputs() -> list[str]:
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def source_digest() -> str:
    """SHA-256 of every input's bytes and of the compiler flags: a library built from other
    sources (or a pushed library newer than its sources) is rebuilt, whatever the mtimes say."""
    h = hashlib.sha256()
    h.update(" ".join(ARCH + COMPILE_FLAGS + LINK_FLAGS).encode())
    for p in inputs():
        h.update(b"\0" + os.path.relpath(p, ROOT).encode() + b"\0")
        with open(p, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def _digest_file(lib: str) -> str:
    return lib + ".sha256"


def stale(lib: str = LIBRARY) -> bool:
    """True unless ``lib`` exists and was built from exactly the current sources and flags."""
    if not os.path.exists(lib) or not os.path.exists(_digest_file(lib)):
        return True
    with open(_digest_file(lib)) as fh:
        return fh.read().strip() != source_digest()


def _run(cmd: list[str]) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(os.path.basename(cmd[0]) + " failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)


@contextlib.contextmanager
def _alone():
    """One process at a time builds in this directory (several ranks make their first call together)."""
    fd = os.open(PKG, os.O_RDONLY)
    try:
        with contextlib.suppress(OSError):  # a file system without locks: the replacements below are atomic all the same
            fcntl.flock(fd, fcntl.LOCK_EX)
        yield
    finally:
        os.close(fd)


def _install(tmp: str, lib: str, digest: str) -> None:
    """Put a built file and its digest in place, each atomically."""
    fd, note = tempfile.mkstemp(suffix=".sha256", dir=PKG)
    with os.fdopen(fd, "w") as fh:
        fh.write(digest + "\n")
    os.chmod(note, 0o644)
    os.replace(tmp, lib)
    os.replace(note, _digest_file(lib))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ (in parallel, one object each) and link them into one
    shared library (atomic replace), unless it is there and up to date."""
    if force or stale(LIBRARY):
        with _alone():
            if force or stale(LIBRARY):  # another process may have built it meanwhile
                _build_library(verbose)
    return LIBRARY


def _build_library(verbose: bool) -> None:
    digest, compiler = source_digest(), nvcc()
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=PKG)
    os.close(fd)
    objdir = tempfile.mkdtemp(prefix="dcp_build_")
    srcs = sources()
    objs = [os.path.join(objdir, os.path.basename(src) + ".o") for src in srcs]
    compiles = [[compiler, *ARCH, *COMPILE_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
                for src, obj in zip(srcs, objs)]
    link = [compiler, *ARCH, *LINK_FLAGS, "-o", tmp, *objs]
    try:
        with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
            for f in [ex.submit(_run, c) for c in compiles]:
                f.result()
        _run(link)
        if verbose:
            for c in compiles + [link]:
                print(" ".join(c))
        _install(tmp, LIBRARY, digest)
    finally:
        if os.path.exists(tmp):
            os.unlink(tmp)
        shutil.rmtree(objdir, ignore_errors=True)


def _build_binding() -> None:
    import torch

    digest = binding_digest()
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=PKG)
    os.close(fd)
    cmd = [os.environ.get("CXX", "g++"), *BINDING_FLAGS,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", os.path.join(base, "include"), "-I", os.path.join(base, "include/torch/csrc/api/include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), BINDING_SOURCE,
           "-L", os.path.join(base, "lib"), *BINDING_LIBS, "-o", tmp]
    try:
        _run(cmd)
        _install(tmp, BINDING, digest)
    finally:
        if os.path.exists(tmp):
            os.unlink(tmp)


def binding_digest() -> str:
    """SHA-256 of the binding's sources and of the compiler flags, the Python and the torch it is built for."""
    import torch

    h = hashlib.sha256()
    h.update(f"{sys.version} {torch.__version__} {' '.join(BINDING_FLAGS + BINDING_LIBS)}".encode())
    for p in (BINDING_SOURCE, *sorted(glob.glob(os.path.join(INCLUDE, "*.h")))):
        with open(p, "rb") as fh:
            h.update(b"\0" + fh.read())
    return h.hexdigest()


def binding_stale() -> bool:
    """True unless the binding exists and was built from exactly the current sources, flags and versions."""
    if not os.path.exists(BINDING) or not os.path.exists(_digest_file(BINDING)):
        return True
    with open(_digest_file(BINDING)) as fh:
        return fh.read().strip() != binding_digest()


def build_binding(force: bool = False) -> str:
    """Compile the torch binding of the paged calls (atomic replace), unless it is there and up to date."""
    if force or binding_stale():
        with _alone():
            if force or binding_stale():
                _build_binding()
    return BINDING


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=True))
    print(build_binding(force=args.force))

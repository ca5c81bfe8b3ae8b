"""Compile libbitlin.so (the C-ABI library) in-tree for sm_103a, and the compiled binding.

Each CUDA source is compiled in parallel with nvcc, then linked into
``hadamard_rotated_binary_gb300/libbitlin.so``; csrc/paged_native.cpp, which takes torch tensors,
is compiled with g++ against the installed torch, if there is one, and linked into
``_paged_native.so`` beside it.
Usage: ``python -m
hadamard_rotated_binary_gb300.build``.
"""
from __future__ import annotations

import glob
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbitlin.so")
NATIVE = os.path.join(PKG, "_paged_native.so")
NATIVE_SRC = os.path.join(CSRC, "paged_native.cpp")
BUILD_DIR = os.path.join(PKG, "_build")
NATIVE_OBJ = os.path.join(BUILD_DIR, "paged_native.o")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libbitlin.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _fingerprint() -> str:
    h = hashlib.sha256()
    files = _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(INCLUDE, "bitlin.h")]
    for f in files:
        with open(f, "rb") as fh:
            h.update(f.encode())
            h.update(fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS).encode())
    h.update(os.uname().machine.encode())
    return h.hexdigest()


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec and spec.submodule_search_locations else None


def _start_native(force: bool):
    """Start compiling paged_native.cpp if it is out of date: (process, fingerprint), or None.
    Where there is no torch there is nothing to bind: the library alone is built."""
    torch = _torch_dir()
    if torch is None:
        return None
    h = hashlib.sha256()
    for f in (NATIVE_SRC, os.path.join(INCLUDE, "bitlin.h"), os.path.join(torch, "version.py")):
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update((sys.version + os.uname().machine).encode())
    fp, stamp = h.hexdigest(), NATIVE + ".stamp"
    if not force and os.path.exists(NATIVE) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == fp:
                return None
    os.makedirs(BUILD_DIR, exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-I{INCLUDE}", f"-I{sysconfig.get_paths()['include']}",
           "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"), f"-I{cuda}", "-c", NATIVE_SRC,
           "-o", NATIVE_OBJ]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), fp


def _finish_native(started) -> None:
    """Link it against libbitlin.so, which it finds beside itself."""
    if started is None:
        return
    proc, fp = started
    out, _ = proc.communicate()
    if proc.returncode != 0:
        sys.stderr.write(out.decode(errors="replace"))
        raise RuntimeError("g++ failed on paged_native.cpp")
    tmp = NATIVE + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", "-o", tmp, NATIVE_OBJ, f"-L{PKG}", "-l:libbitlin.so", "-Wl,-rpath,$ORIGIN",
                    f"-L{os.path.join(_torch_dir(), 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"],
                   check=True)
    os.replace(tmp, NATIVE)
    with open(NATIVE + ".stamp", "w") as f:
        f.write(fp)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libbitlin.so and, where torch is installed, the compiled binding, if their sources
    changed (or force); returns the library's path."""
    started = _start_native(force)
    try:
        path = _build_library(force, verbose)
    except BaseException:
        if started is not None:
            started[0].kill()
            started[0].communicate()
        raise
    _finish_native(started)
    return path


def _build_library(force: bool, verbose: bool) -> str:
    stamp = LIB + ".stamp"
    fp = _fingerprint()
    if not force and os.path.exists(LIB) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == fp:
                return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [cc] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    errors = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            errors.append(src)
    if errors:
        raise RuntimeError("nvcc failed on: " + ", ".join(os.path.basename(e) for e in errors))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([cc] + ARCH + ["-shared", "-o", tmp] + objs, check=True)
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(fp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

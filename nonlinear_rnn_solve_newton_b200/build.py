"""Build libpararnn.so in-tree with nvcc for sm_100a (B200)."""
from __future__ import annotations

import glob
import hashlib
import os
import re
import shutil
import subprocess
import sys
import time

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libpararnn.so")
BUILD = os.path.join(HERE, "_build")  # objects, kept for the next build
SOURCES = [os.path.join(CSRC, f) for f in ("pararnn.cu", "linattn.cu", "norm.cu")]
DEPS = SOURCES + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [
    os.path.join(INCLUDE, "pararnn.h"), os.path.abspath(__file__)]


def nvcc_path() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libpararnn.so")
    return cand


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in DEPS)


def _includes(path, seen=None):
    """The file and the project files it includes, directly or not."""
    seen = set() if seen is None else seen
    if path not in seen:
        seen.add(path)
        with open(path, encoding="utf-8") as f:
            names = re.findall(r'^\s*#include\s+"([^"]+)"', f.read(), flags=re.M)
        for n in names:
            for d in (CSRC, INCLUDE):
                if os.path.exists(os.path.join(d, n)):
                    _includes(os.path.join(d, n), seen)
    return seen


def _flags():
    return ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
            "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _settings(flags):
    """A name for what makes an object besides its sources: the flags and the compiler."""
    version = subprocess.run([nvcc_path(), "--version"], capture_output=True, check=True).stdout
    return hashlib.sha256(repr(flags).encode() + version).hexdigest()[:12]


def _object(src, settings):
    return os.path.join(BUILD, f"{os.path.basename(src)}.{settings}.o")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    # Results are as old as the start of the build that made them: a source edited while it
    # is compiled is newer, and compiled again.
    started = time.time_ns()
    own = f".{os.getpid()}.tmp"  # two processes may build at once
    flags = _flags()
    settings = _settings(flags)

    def put(path):
        os.utime(path + own, ns=(started, started))
        os.replace(path + own, path)

    os.makedirs(BUILD, exist_ok=True)
    jobs = []
    for src in SOURCES:  # the sources that changed, side by side
        obj = _object(src, settings)
        if not force and os.path.exists(obj):
            t = os.path.getmtime(obj)
            if all(os.path.getmtime(p) <= t for p in _includes(src)):
                continue
        cmd = [nvcc_path(), *(["-Xptxas=-v"] if verbose else []), *flags, "-c", src, "-o", obj + own]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        jobs.append((cmd, obj, subprocess.Popen(cmd)))
    failed = None
    for cmd, obj, job in jobs:
        rc = job.wait()
        if rc == 0:
            put(obj)
        else:
            failed = failed or subprocess.CalledProcessError(rc, cmd)
    if failed:
        raise failed
    subprocess.check_call([nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                           *[_object(s, settings) for s in SOURCES], "-o", LIB + own])
    put(LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)

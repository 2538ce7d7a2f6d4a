"""Build libpararnn.so in-tree with nvcc for sm_100a (B200)."""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libpararnn.so")
SOURCES = [os.path.join(CSRC, f) for f in ("pararnn.cu", "linattn.cu", "norm.cu")]
DEPS = SOURCES + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(INCLUDE, "pararnn.h")]


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


def _object(src):
    return os.path.join(HERE, "_build", os.path.basename(src) + ".o")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
             "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]
    if verbose:
        flags.insert(0, "-Xptxas=-v")
    os.makedirs(os.path.join(HERE, "_build"), exist_ok=True)
    jobs = []
    for src in SOURCES:  # the sources that changed, side by side
        obj = _object(src)
        if not force and os.path.exists(obj):
            t = os.path.getmtime(obj)
            if all(os.path.getmtime(p) <= t for p in _includes(src)):
                continue
        cmd = [nvcc_path(), *flags, "-c", src, "-o", obj + ".tmp"]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        jobs.append((cmd, obj, subprocess.Popen(cmd)))
    failed = None
    for cmd, obj, job in jobs:
        rc = job.wait()
        if rc == 0:
            os.replace(obj + ".tmp", obj)
        else:
            failed = failed or subprocess.CalledProcessError(rc, cmd)
    if failed:
        raise failed
    subprocess.check_call([nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                           *[_object(s) for s in SOURCES], "-o", LIB + ".tmp"])
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)

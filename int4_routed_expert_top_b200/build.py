"""Build libcolimoe.so in-tree with nvcc for sm_100a.

    python -m int4_routed_expert_top_b200.build
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libcolimoe.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-ffp-contract=off",
    "--expt-relaxed-constexpr",
]

# translation units, linked into one library
UNITS = ("coli_moe", "block", "fp4")


def sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")) +
                  glob.glob(os.path.join(PKG, "csrc", "*.cuh")) +
                  [os.path.join(ROOT, "include", "coli_moe.h")])


def unit_sources(unit: str):
    """The unit's .cu file and every header of this repository that it includes."""
    todo, seen = [os.path.join(PKG, "csrc", unit + ".cu")], set()
    while todo:
        path = todo.pop()
        if path in seen:
            continue
        seen.add(path)
        with open(path) as f:
            names = re.findall(r'^#include "(\w+\.c?u?h)"', f.read(), re.M)
        for name in names:
            for folder in (os.path.join(PKG, "csrc"), os.path.join(ROOT, "include")):
                if os.path.exists(os.path.join(folder, name)):
                    todo.append(os.path.join(folder, name))
    return sorted(seen)


def _older(target: str, files) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in files)


def stale() -> bool:
    return _older(LIB, sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    objects, running = [], []
    for unit in UNITS:  # stale units side by side
        obj = os.path.join(PKG, "csrc", unit + ".o")
        objects.append(obj)
        if not force and not _older(obj, unit_sources(unit)):
            continue
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [NVCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(PKG, "csrc", unit + ".cu"), "-o", tmp]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        running.append((subprocess.Popen(cmd), cmd, tmp, obj))
    codes = [(p.wait(), cmd, tmp, obj) for p, cmd, tmp, obj in running]
    for rc, cmd, tmp, obj in codes:
        if rc != 0:
            raise subprocess.CalledProcessError(rc, cmd)
        os.replace(tmp, obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, *FLAGS, "-shared", *objects, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

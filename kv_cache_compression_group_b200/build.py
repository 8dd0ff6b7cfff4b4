"""Build libjolt.so (the sm_100a C-ABI library) in-tree with nvcc."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libjolt.so")
SOURCES = ["jolt_api.cu", "cache_api.cu", "cache_few_d64.cu", "cache_few_d128.cu",
           "cache_many_d64.cu", "cache_many_d128.cu"]
DEPS = ["jolt_api.cu", "common.cuh", "gemm.cuh", "kernels.cuh", "misc.cuh", "umma.cuh", "eig_cluster.cuh", "chol.cuh",
        "fp16_exact.cuh", "table_tc.cuh", "attend.cuh", "eig_large.cuh", "host.cuh", "cache_api.cu", "cache.cuh", "cache_split.cuh",
        "cache_attend.cuh", "cache_attend_codes.cuh", "cache_attend_tc.cuh", "cache_launch.cuh",
        "cache_few_d64.cu", "cache_few_d128.cu", "cache_many_d64.cu", "cache_many_d128.cu"]
CACHE = [d for d in DEPS if d.startswith("cache") and d.endswith(".cuh")]


def nvcc_cmd(source: str, out: str, extra=()) -> list:
    return (["nvcc", "-std=c++17", "-O3", "-lineinfo",
             "-gencode", "arch=compute_100a,code=sm_100a",
             "-Xcompiler", "-fPIC", "-c",
             "-I", os.path.join(ROOT, "include"),
             "-o", out, os.path.join(CSRC, source)] + list(extra))


def link_cmd(objects: list, out: str) -> list:
    return (["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", out] + objects + ["-lcusolver"])


def _newer(target: str, paths) -> bool:
    """Whether target exists and is no older than any of paths."""
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in paths)


def _inputs(source: str) -> list:
    """Files whose change rebuilds a source's object: all headers, but the cache's own for the cache alone."""
    headers = [d for d in DEPS if d.endswith(".cuh") and (d not in CACHE or source.startswith("cache"))]
    return [os.path.join(CSRC, d) for d in [source] + headers] + [os.path.join(ROOT, "include", "jolt.h")]


def up_to_date() -> bool:
    return _newer(LIB, [os.path.join(CSRC, d) for d in DEPS] + [os.path.join(ROOT, "include", "jolt.h")])


def build(force: bool = False, verbose: bool = True) -> str:
    """Compile the sources that changed (side by side) and link the library."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    running, objects = [], []
    for source in SOURCES:
        obj = os.path.join(OBJ, source.replace(".cu", ".o"))
        objects.append(obj)
        if not force and _newer(obj, _inputs(source)):
            continue
        cmd = nvcc_cmd(source, obj + ".tmp")
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        running.append((obj, cmd, subprocess.Popen(cmd)))
    for obj, cmd, p in running:
        if p.wait() != 0:
            raise subprocess.CalledProcessError(p.returncode, cmd)
        os.replace(obj + ".tmp", obj)
    tmp = LIB + ".tmp"
    subprocess.run(link_cmd(objects, tmp), check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv)

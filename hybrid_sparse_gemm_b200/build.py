"""Build libpatch_hybrid.so (the C-ABI library) in-tree with nvcc for sm_100a,
and _binding.<interpreter>.so (the Python argument marshalling of its 8-bit calls)
with gcc.

    python -m hybrid_sparse_gemm_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libpatch_hybrid.so")
# named for the interpreter it is built for: another one looks for its own
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CC = os.environ.get("CC", "gcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--shared", "--threads", "0",
    "-Xptxas", "-v",
]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def stale(out: str, inputs) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(f) > t for f in [*inputs, __file__])


def _run(cmd, out: str, what: str, verbose: bool):
    r = subprocess.run([*cmd, "-o", out + ".tmp"], capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + r.stderr[-6000:])
    os.replace(out + ".tmp", out)


def build(force: bool = False, verbose: bool = False) -> str:
    include = os.path.join(ROOT, "include")
    binding = os.path.join(HERE, "csrc", "binding.c")
    if force or stale(LIB, sources() + headers()):
        _run([NVCC, *FLAGS, "-I", include, "-I", os.path.join(HERE, "csrc"), *sources()], LIB, "nvcc", verbose)
    if force or stale(BINDING, [binding] + headers()):
        _run([CC, "-O2", "-Wall", "-shared", "-fPIC", "-I", include, "-I", sysconfig.get_paths()["include"], binding],
             BINDING, CC, verbose)
    untagged = os.path.join(HERE, "_binding.so")  # of an earlier build: any interpreter would load it
    if os.path.exists(untagged) and untagged != BINDING:
        os.remove(untagged)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)

"""Build libkda.so in-tree with nvcc for sm_100a (B200)."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkda.so")
ROOT = os.path.dirname(HERE)

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-v",
]
# translation units, compiled at the same time
UNITS = ["kda_lib.cu", "kda_norm.cu", "kda_conv.cu", "kda_scan.cu", "kda_scan_bwd.cu"]


def _sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh"))] + [
        os.path.join(ROOT, "include", "kda.h")]


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, u + ".o") for u in UNITS]
        runs = [subprocess.Popen([nvcc, *NVCC_FLAGS, "-c", "-I", os.path.join(ROOT, "include"), "-o", o, os.path.join(CSRC, u)],
                                 stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for u, o in zip(UNITS, objs)]
        logs = [r.communicate()[0] for r in runs]
        for u, r, log in zip(UNITS, runs, logs):
            if r.returncode != 0:
                sys.stderr.write(log)
                raise RuntimeError(f"nvcc failed building {u}")
        if verbose:
            sys.stderr.write("".join(logs))
        lib = LIB + ".tmp%d" % os.getpid()
        subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", lib, *objs], check=True)
        os.replace(lib, LIB)
    with open(os.path.join(HERE, "ptxas_info.txt"), "w") as f:
        f.write("".join(logs))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)

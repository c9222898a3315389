"""Build libzero.so (the gfx950 HIP kernels and the C ABI) in-tree with hipcc."""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libzero.so")
SOURCES = ["abi.cpp", "layout.cpp", "step_kernels.hip", "gather_kernels.hip", "layer_abi.cpp",
           "linear_kernels.hip", "dropout_kernels.hip"]
# host-only C++ (no device pass), compiled to an object and linked in
HOST_SOURCES = ["offload.cpp"]
HOST_FLAGS = ["-x", "c++", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-Wall", "-c"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off",                                   # one rounding per source operation
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "hipcc"


def _run(cmd):
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + " ".join(cmd) + "\n" + proc.stdout + proc.stderr)


def build(out: str = LIB, extra=()) -> str:
    """Compile every source into ``out`` (always recompiles, a few sources at a time)."""
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(hipcc()) or hipcc())))
    jobs, objs = [], []
    for s in SOURCES + HOST_SOURCES:
        obj = out + "." + os.path.splitext(s)[0] + ".o"
        objs.append(obj)
        if s in HOST_SOURCES:
            jobs.append([hipcc(), *HOST_FLAGS, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                         *inc, os.path.join(CSRC, s), "-o", obj])
        else:
            flags = [f for f in HIPCC_FLAGS if f != "-shared"]
            jobs.append([hipcc(), *flags, *extra, *inc, "-c", os.path.join(CSRC, s), "-o", obj])
    try:
        with ThreadPoolExecutor(max_workers=4) as pool:
            list(pool.map(_run, jobs))
        _run([hipcc(), "--offload-arch=gfx950", "-fPIC", "-shared", *objs, "-o", out + ".tmp"])
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    os.replace(out + ".tmp", out)
    return out


if __name__ == "__main__":
    print(build())

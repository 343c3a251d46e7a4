"""Build libconvt.so (the HIP library for gfx950) in place with hipcc.

Run as ``python -m convt_forward_amd.build`` or through ``__graft_entry__.build()``.
Every call recompiles every source.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libconvt.so")
BUILD_DIR = os.path.join(HERE, "_build")

SOURCES = ["plan.cpp", "api.cpp", "k_misc.hip", "k_phase_gemm.hip", "k_gemm_nchw.hip", "k_gemm_allphase.hip",
           "k_bwd_allphase.hip", "k_bwd_grouped.hip", "k_grouped.hip", "noalloc.hip",
           "decode_api.cpp", "k_rms_norm.hip", "k_cache.hip", "k_attend.hip", "k_attend_mfma.hip",
           "k_q4_matvec.hip", "k_q4_mfma.hip"]

# Packed-FP32 instructions are kept out of every kernel (the target feature is
# switched off for the device pass; the host pass ignores it with a warning).
HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + INCLUDE, "-I" + CSRC,
]


# Per-source device flags. The grouped kernel keeps its MFMA accumulators in
# ordinary VGPRs (no AGPR copies around its short MFMA chains).
SOURCE_FLAGS = {
    "k_grouped.hip": ["-Xarch_device", "-mllvm=-amdgpu-mfma-vgpr-form"],
}


def _hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [_hipcc()] + HIP_FLAGS + SOURCE_FLAGS.get(src, []) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "'-packed-fp32-ops' is not a recognized feature for this target (ignoring feature)"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [_hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)

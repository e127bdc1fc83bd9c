"""Build libqgemm.so (gfx950) in-tree with hipcc.

Usage: python -m weight_only_quantized_w8a16_amd.build
Each source compiles to an object under _build/ in parallel, then the objects
are linked into weight_only_quantized_w8a16_amd/libqgemm.so.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libqgemm.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
DEVICE_SOURCES = ["transform.hip", "decode.hip", "prefill.hip", "moe.hip", "w8a8.hip", "embed.hip", "mx4.hip", "mx4_gemm.hip",
                  "f8.hip", "f8_gemm.hip", "probe.hip"]
HOST_SOURCES = ["api.cpp", "override.cpp"]
COMMON = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function"]
# Packed fp32 VALU ops disabled: plain float code must not be turned into
# v_pk_{add,mul,fma}_f32.
# A launch bound or an unrolling that the compiler cannot keep is an error:
# host code and comments reckon with what the kernels ask for.
DEVICE_FLAGS = [f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang",
                "-packed-fp32-ops", "-munsafe-fp-atomics", "-Werror=pass-failed"]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON]
    if src.endswith(".hip"):
        cmd += DEVICE_FLAGS
    else:
        cmd += ["-D__HIP_PLATFORM_AMD__"]
    cmd += ["-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{res.stderr}")
    # Warnings, but for the host pass's about the device's feature.
    said = [ln for ln in res.stderr.splitlines() if ln.strip() and not ln.startswith("'-packed-fp32-ops'")]
    if said:
        print(f"hipcc on {src}:", *said, sep="\n", file=sys.stderr, flush=True)
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = DEVICE_SOURCES + HOST_SOURCES
    with ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)

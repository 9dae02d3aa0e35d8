"""Builds liboidn_mi355x.so in-tree with hipcc for gfx950.

Usage: python -m unet_x3_convolution_amd.build   (or call build()).
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig
from importlib.machinery import EXTENSION_SUFFIXES

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "liboidn_mi355x.so")
BINDING = os.path.join(HERE, "_binding" + EXTENSION_SUFFIXES[0])      # of this Python's ABI
SOURCES = ["api.cpp", "conv_f16.hip", "conv_f32.hip", "elementwise.hip", "noalloc.hip",
           "calibrate.hip", "dense_api.cpp", "dense_rows.hip", "dense_gemm16_forward.hip",
           "dense_gemm16_gated_back.hip", "dense_gemm16_group.hip", "dense_gemm32.hip", "dense_few.hip", "dense_narrow.hip",
           "norm_api.cpp", "norm.hip", "norm_back.hip", "fp8_api.cpp", "fp8_rows.hip", "fp8_gemm.hip",
           "fp8_few.hip", "fp8_narrow.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ROCM_INCLUDE = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")
PYTHON_INCLUDE = sysconfig.get_paths()["include"]
# Packed-fp32 ops are turned off for the device code: plain fp32 arithmetic only.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include")]


# Per-source options: the MFMA calibration stream keeps its accumulators in
# arch VGPRs (in accumulation registers the compiler shuffled them between
# loop iterations).
SOURCE_FLAGS = {"calibrate.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


def _compile(src: str) -> str:
    obj = os.path.join(OBJ_DIR, src + ".o")
    cmd = [HIPCC, *FLAGS, *SOURCE_FLAGS.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _binding() -> None:
    """The Python calls of csrc/binding.cpp, on the library beside them.  Without Python's headers there
    are none, and the package calls the library through ctypes, which takes more of the host's time."""
    if not os.path.exists(os.path.join(PYTHON_INCLUDE, "Python.h")):
        sys.stderr.write(f"no Python.h in {PYTHON_INCLUDE}: {os.path.basename(BINDING)} is not built, "
                         "its calls go through ctypes\n")
        if os.path.exists(BINDING):      # an earlier library's
            os.remove(BINDING)
        return
    tmp = BINDING + ".tmp"
    # host code alone; the HIP runtime is the library's
    cmd = [HIPCC, "-x", "c++", "-no-hip-rt", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
           "-I", PYTHON_INCLUDE, "-isystem", ROCM_INCLUDE, os.path.join(CSRC, "binding.cpp"),
           "-L", HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"building the binding failed:\n{res.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = True) -> str:
    os.makedirs(OBJ_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    _binding()
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()

"""Build the gfx950 HIP library libbsfp8.so in-tree with hipcc (cross-compiles without a GPU), and the
binding's C part _calls with the host's C compiler, where there is one and Python's headers: without it
the calls go through ctypes.

    python -m blockwise_scaled_fp8_act_amd.build
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libbsfp8.so")
# named for this interpreter, whose full C interface it uses: another one does not load it
CALLS_PATH = os.path.join(PKG, "_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

SOURCES = ["capi.cpp", "quantize.hip", "gemm.hip", "moe.hip", "gemm_routed.hip", "norm.hip", "swiglu.hip", "quantize_i8.hip", "gemm_i8.hip",
           "grads.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CC = os.environ.get("CC", "gcc")
ARCH = "gfx950"
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # keep the compiler from forming packed-fp32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results in VGPRs: the GEMM rescales every partial product with VALU FMAs
    "-mllvm", "-amdgpu-mfma-vgpr-form=1",
    "-Wall", "-Wno-unused-function",
    "-I", INCLUDE, "-I", CSRC,
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _build_calls() -> bool:
    """False: left out. Whatever an earlier build made is gone then, so that none outlives the library's
    signatures it was compiled for."""
    include, tmp = sysconfig.get_paths()["include"], CALLS_PATH + ".tmp"
    made = shutil.which(CC) is not None and os.path.exists(os.path.join(include, "Python.h"))
    if made:
        cmd = [CC, "-O2", "-std=gnu11", "-fPIC", "-shared", "-Wall", "-I", INCLUDE, "-I", include, os.path.join(CSRC, "calls.c"), "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{CC} failed for calls.c:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, CALLS_PATH)
    for old in glob.glob(os.path.join(PKG, "_calls*.so")):
        if not (made and old == CALLS_PATH):
            os.remove(old)
    return made


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link libbsfp8.so, compile _calls (always recompiles)."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    calls = _build_calls()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(f"built {LIB_PATH}")
        print(f"built {CALLS_PATH}" if calls else "no C compiler or no Python.h: calls go through ctypes alone")
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)

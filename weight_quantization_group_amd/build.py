"""Build the HIP libraries ``libhqq.so`` and ``libhqq_layers.so`` for gfx950, in-tree.

    python -m weight_quantization_group_amd.build

The translation units are compiled in parallel (one hipcc process each) and
linked into one shared library per header of include/.  Flags that matter for exactness:
  -ffp-contract=off                  no fma contraction beyond the explicit ones
  -fno-gpu-flush-denormals-to-zero   fp32 denormals kept (IEEE)
  (HIP's default fp32 division is correctly rounded; no unsafe-math flags)
  -Xclang -target-feature -Xclang -packed-fp32-ops   no packed-fp32 VALU ops
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libhqq.so")

SOURCES = ["hqq_abi.cpp", "hqq_stream.cpp", "hqq_solve.hip", "hqq_solve_b1.hip", "hqq_solve_b2.hip",
           "hqq_solve_b3.hip", "hqq_solve_b4.hip", "hqq_solve_b8.hip",
           "hqq_solve_b1_bf16.hip", "hqq_solve_b2_bf16.hip", "hqq_solve_b3_bf16.hip",
           "hqq_solve_b4_bf16.hip", "hqq_solve_b8_bf16.hip", "hqq_codec.hip",
           "hqq_linear.hip", "hqq_gemm.cpp"]

LAYERS_LIB = os.path.join(PKG, "libhqq_layers.so")
LAYERS_SOURCES = ["hqq_layers_abi.cpp", "hqq_layers_unpack.hip", "hqq_layers_gemm.hip", "hqq_layers_rows.hip",
                  "hqq_layers_skinny_one.hip", "hqq_layers_skinny_pair.hip", "hqq_layers_skinny_grad.hip"]

FLAGS = ["-O3", "--offload-arch=gfx950", "-std=c++17", "-fPIC", "-fvisibility=hidden",
         "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wno-pass-failed",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = ["hipcc", *FLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _link(lib: str, objs, libs=()) -> None:
    tmp = lib + ".tmp"
    cmd = ["hipcc", "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs, *libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    todo = SOURCES + LAYERS_SOURCES
    with cf.ThreadPoolExecutor(max_workers=len(todo)) as ex:
        objs = dict(zip(todo, ex.map(_compile, todo)))
    _link(LIB, [objs[s] for s in SOURCES], ["-lhipblaslt"])
    _link(LAYERS_LIB, [objs[s] for s in LAYERS_SOURCES])
    if verbose:
        print("built", LIB)
        print("built", LAYERS_LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)

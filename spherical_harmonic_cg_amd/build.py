"""Build step for the HIP library: compiles csrc/*.hip for gfx950 and links
spherical_harmonic_cg_amd/libeqtp.so in-tree.

Usage: python -m spherical_harmonic_cg_amd.build [--jobs N]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libeqtp.so")
ROOT = os.path.dirname(HERE)

SOURCES = ["abi.hip", "sh.hip", "sort.hip", "conv_node.hip", "conv_edge.hip", "conv_bwd.hip", "conv_so2.hip", "conv_bwd_so2.hip", "linear.hip", "interaction.hip", "check.hip", "norm.hip", "norm_grad.hip",
           "dropout.hip", "attention.hip", "abi_block.hip", "distance_bias.hip", "head_norm.hip", "route.hip",
           "expert_plan.hip", "expert.hip", "expert_grad.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # packed fp32 instructions are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-I", CSRC,
]


# per-source additions: the radial edge-aligned kernel and the grad_vec kernel
# consume their matrix-core results on the vector ALUs, so they are produced in
# VGPRs (no copies out of the accumulation registers); the experts' weight
# gradient, too, which then holds 150 to 168 registers instead of 124 and 64 (three
# waves a SIMD, not two; bf16 under gates 177 to 193)
EXTRA_FLAGS = {"conv_so2.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
               "conv_bwd.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
               "expert_grad.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src.replace(".hip", ".o"))
    cmd = [HIPCC] + FLAGS + EXTRA_FLAGS.get(src, []) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, out))
    return obj


def build(jobs: int = 8, verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(jobs, len(SOURCES)))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=8)
    args = ap.parse_args()
    build(args.jobs)
    sys.exit(0)

"""Build the HIP library (gfx950) and the CPU check library, in-tree.

    python -m bit_gemm_amd.build

produces bit_gemm_amd/libmosaicq.so (the C ABI of include/mosaicq.h),
bit_gemm_amd/libmosaicq_block.so (the C ABI of include/mosaicq_block.h),
bit_gemm_amd/libmosaicq_head.so (the C ABI of include/mosaicq_head.h) and
bit_gemm_amd/libmq_hostcheck.so (the packer's integer arithmetic built for
the host, used by CPU tests). Every call recompiles.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmosaicq.so")
BLOCK_LIB = os.path.join(HERE, "libmosaicq_block.so")
HEAD_LIB = os.path.join(HERE, "libmosaicq_head.so")
HOSTCHECK = os.path.join(HERE, "libmq_hostcheck.so")
SOURCES = ["api.cpp", "pack.hip", "pack_blocks.hip", "gemv.hip", "gemm.hip", "gemm_mid.hip", "gemm_rw.hip", "residual.hip", "migrate.hip", "w4a4.hip", "probe.hip"]
BLOCK_SOURCES = ["block_api.cpp", "rope.hip", "norm.hip", "kv_append.hip", "kv_attn.hip", "kv_attn_rows.hip"]
HEAD_SOURCES = ["head_api.cpp", "quantize8.hip", "linear8.hip", "sample.hip"]
# per-source code generation options: the prefill GEMM's stage body is one
# long basic block; the ILP-oriented machine scheduler interleaves its
# widening arithmetic with the MFMAs instead of clustering it after them
EXTRA: dict = {"gemm.hip": ["-mllvm", "-amdgpu-sched-strategy=max-ilp"]}
ARCH = os.environ.get("MQ_OFFLOAD_ARCH", "gfx950")


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _flags():
    return ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-fvisibility=hidden",
            # packed fp32 VALU forms are kept out of the device code
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError(f"build step failed: {cmd[-1]}")
    return r


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()
    obj_of = {src: os.path.join(BUILD, os.path.splitext(src)[0] + ".o") for src in SOURCES + BLOCK_SOURCES + HEAD_SOURCES}
    cmds = []
    for src, obj in obj_of.items():
        cmds.append([cc, "-x", "hip", *_flags(), *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj])
    with ThreadPoolExecutor(max_workers=min(4, len(cmds))) as ex:
        list(ex.map(_run, cmds))
    for lib, sources in ((LIB, SOURCES), (BLOCK_LIB, BLOCK_SOURCES), (HEAD_LIB, HEAD_SOURCES)):
        tmp = lib + ".tmp"
        _run([cc, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp, *[obj_of[src] for src in sources]])
        os.replace(tmp, lib)
    tmp = HOSTCHECK + ".tmp"
    _run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-I", CSRC,
          os.path.join(CSRC, "hostcheck.cpp"), "-o", tmp])
    os.replace(tmp, HOSTCHECK)
    if verbose:
        print(f"built {LIB}, {BLOCK_LIB}, {HEAD_LIB} and {HOSTCHECK}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)

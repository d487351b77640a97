"""Build the WKV7 HIP library (libwkv7.so) for gfx950 in-tree with hipcc.

Every translation unit is compiled with packed-fp32 instructions disabled;
objects go to ``_build/`` next to this file, the shared library next to the
package so that it travels with the source tree.
"""

from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libwkv7.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["wkv7_api.cpp", "wkv7_seq.hip", "wkv7_chunk_fwd.hip", "wkv7_bwd.hip", "wkv7_static.hip",
           "wkv7_epilogue.hip", "wkv7_chunk128.hip", "wkv7_ssm_api.cpp", "wkv7_ssm.hip",
           "wkv7_ssm_bwd.hip", "wkv7_conv.hip", "wkv7_linattn_api.cpp", "wkv7_linattn.hip",
           "wkv7_linattn_bwd.hip", "wkv7_linattn_rest.hip", "wkv7_gnorm_api.cpp", "wkv7_gnorm.hip", "wkv7_gnorm_bwd_bf16.hip",
           "wkv7_gnorm_bwd_f32.hip",
           "wkv7_slots_api.cpp", "wkv7_slots.hip"]

COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # Matrix-core results stay in ordinary VGPRs (the kernels read every
    # accumulator tile back on the vector ALU; accumulation registers would need
    # a copy instruction per element).
    "-mllvm", "-amdgpu-mfma-vgpr-form=1",
    # Atomics here come from a single lane (work queues, flags); the optimizer's
    # wave-aggregated form reads the result back at once, which makes the issuing
    # wave wait for the atomic's round trip where it is issued.
    "-mllvm", "-amdgpu-atomic-optimizer-strategy=None",
    "-Wno-unused-command-line-argument",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build()

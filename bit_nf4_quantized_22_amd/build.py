"""Build the HIP library libqlora_nf4.so for gfx950, in-tree.

    python -m bit_nf4_quantized_22_amd.build

Compiles every source under csrc/ with hipcc (--offload-arch=gfx950, -O3, no
fast-math, packed fp32 instructions disabled) into _build/, then links
lib/libqlora_nf4.so.  Always rebuilds.
"""

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libqlora_nf4.so")

SOURCES = ["qn_tables.cpp", "qn_api.cpp", "qn_quant.hip", "qn_gemv.hip", "qn_gemm.hip",
           "qn_grads.hip", "qn_merge.hip", "qn_fp8_quant.hip", "qn_fp8_gemm.hip", "qn_fp8_gemv.hip",
           "qn_mx_quant.hip", "qn_mx_gemm.hip", "qn_mx_gemv.hip",
           "qn_optim.hip", "qn_optim_multi.hip", "qn_muon.hip", "qn_dropout.hip",
           "qn_scratch.hip", "qn_probe.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17", "-fvisibility=hidden",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _compile(src, extra=(), build_dir=BUILD):
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC] + FLAGS + list(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    errs = "\n".join(l for l in p.stderr.splitlines()
                     if "packed-fp32-ops" not in l)  # host pass does not know the feature
    if p.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{errs}")
    return obj


def build(verbose=False, extra_flags=(), lib_path=LIB, build_dir=BUILD):
    """Compile and link; extra_flags / lib_path / build_dir allow side builds."""
    os.makedirs(build_dir, exist_ok=True)
    os.makedirs(os.path.dirname(lib_path), exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(6, len(SOURCES))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra_flags, build_dir), SOURCES))
    tmp = lib_path + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stderr}")
    os.replace(tmp, lib_path)
    if verbose:
        print(f"built {lib_path}")
    return lib_path


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)

"""Build of the INSTANT HIP library (gfx950) into this package directory.

``build()`` compiles every source under ``csrc/`` with hipcc for gfx950 and links
``libinstant.so`` next to this file. It always recompiles (the build is the
"does it build" check); objects go to ``<repo>/_build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
REPO = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(REPO, "include")
OUT = os.path.join(HERE, "libinstant.so")
OBJDIR = os.path.join(REPO, "_build")

SOURCES = ["kernels_proj.hip", "kernels_hot.hip", "kernels_gemm.hip", "kernels_calib.hip", "kernels_eig.hip",
           "kernels_linear.hip", "kernels_tile_bf16_fwd.hip", "kernels_tile_bf16_gx.hip", "kernels_tile_bf16_gw.hip",
           "kernels_tile_fp32_fwd.hip", "kernels_tile_fp32_gx.hip", "kernels_tile_fp32_gw.hip",
           "kernels_ckpt.hip", "kernels_norm.hip", "instant_api.cpp", "ops_api.cpp"]

COMMON = ["--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17", "-fvisibility=hidden",
          "-I" + INCLUDE, "-I" + CSRC]
# hipcc flag for the device pass: no packed-fp32 instructions in generated code
DEVICE_ONLY = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the INSTANT library needs ROCm's hipcc")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc()] + COMMON + DEVICE_ONLY + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{msgs}")
    if verbose and msgs.strip():
        print(msgs)
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = OUT + ".tmp"
    cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(verbose=True))

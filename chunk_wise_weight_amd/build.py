"""Build libttt.so (the HIP library behind the C ABI) for gfx950 with hipcc, and the binding's reader of tensor lists
(host code, with g++; where there is none, the binding reads them in Python).

Usage: python -m chunk_wise_weight_amd.build [--verbose]
Both are written next to this file, in-tree.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libttt.so")
# the binding's own extension module: reads what it needs of a list of tensors in one pass
LISTS_SRC = os.path.join(CSRC, "tensor_lists.cpp")
LISTS = os.path.join(PKG, "_tensor_lists.so")
# a standalone program: MFMA throughput and shader clock under the power limit (not part of the library)
PROBE_SRC = os.path.join(PKG, "probes", "mfma_clock.hip")
PROBE = os.path.join(PKG, "probes", "mfma_clock")
SOURCES = ["ttt_api.hip", "kernels_bf16.hip", "kernels_f32.hip", "kernels_clip.hip", "kernels_target.hip", "kernels_misc.hip",
           "block_api.hip", "kernels_norm.hip", "kernels_embed.hip", "kernels_grads.hip",
           "dense_api.hip", "kernels_linear.hip", "kernels_dense.hip", "kernels_few.hip",
           "kernels_adamw.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # keep fp32 arithmetic on scalar/vector FMA forms, not packed-fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-result",
]


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; the ROCm toolchain is required to build libttt.so")


def _build_lists(verbose: bool) -> bool:
    """The native list reader. Where it cannot be built (no host compiler, no Python headers) the binding reads lists in
    Python; what an earlier build left is then removed."""
    import torch

    from .binding import built_for

    at = os.path.dirname(torch.__file__)
    inc = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", *[f"-I{i}" for i in inc],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DBUILT_FOR="{built_for()}"', LISTS_SRC,
           "-o", LISTS + ".tmp", f"-L{os.path.join(at, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = r.returncode != 0 and f"{r.stdout}\n{r.stderr}"
    except OSError as e:
        failed = str(e)
    if failed:
        if os.path.exists(LISTS):
            os.remove(LISTS)
        warnings.warn(f"{cmd[0]} failed on {LISTS_SRC}; lists of tensors will be read in Python:\n{failed}", RuntimeWarning)
        return False
    os.replace(LISTS + ".tmp", LISTS)
    return True


def build(verbose: bool = False) -> str:
    hipcc = _hipcc()
    os.makedirs(OBJDIR, exist_ok=True)
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
        cmd = [hipcc, *HIPCC_FLAGS, *inc, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(4, len(SOURCES))) as ex:
        lists = ex.submit(_build_lists, verbose)
        objs = list(ex.map(compile_one, SOURCES))
        lists.result()
    tmp = LIB + ".tmp"
    cmd = [hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    cmd = [hipcc, *[f for f in HIPCC_FLAGS if f != "-fPIC"], "-o", PROBE + ".tmp", PROBE_SRC]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {PROBE_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(PROBE + ".tmp", PROBE)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))

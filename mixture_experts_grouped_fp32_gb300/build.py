"""Build ``libmoe.so`` in-tree: each ``csrc/*.cu`` compiled for sm_103a in parallel, then linked.

    python -m mixture_experts_grouped_fp32_gb300.build [--verbose]

The CUDA runtime is linked statically, and the driver's tensor-map encoder is reached through
``cudaGetDriverEntryPointByVersion``, so the library loads on a machine without a GPU driver
(its entry points then return MOE_ERR_CUDA).

Beside it, ``_moe_fast.so``: the binding's usual calls without Python's share of their cost (g++ against
torch's headers).  Its functions only forward to ``libmoe.so``; where it cannot be built the binding
works without it.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libmoe.so")
FAST = os.path.join(HERE, "_moe_fast.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _compile(src: str, verbose: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr


def _build_fast() -> str:
    """Compiles the fast binding; returns why not if it cannot be."""
    import torch
    t = os.path.dirname(torch.__file__)
    tmp = FAST + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DMOE_TORCH_VERSION="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + os.path.join(t, "include"),
           "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda",
           "-lc10", "-lc10_cuda", "-ldl"]
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return str(e)
    if res.returncode != 0:
        return res.stderr
    os.replace(tmp, FAST)
    return ""


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        fast = ex.submit(_build_fast)
        results = list(ex.map(lambda s: _compile(s, verbose), srcs))
        why = fast.result()
    if why:
        if os.path.exists(FAST):
            os.remove(FAST)  # an older one could expect another library
        sys.stderr.write(f"_moe_fast.so was not built (the binding works without it):\n{why[-2000:]}\n")
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true", help="print ptxas resource usage")
    print(build(ap.parse_args().verbose))

"""Compile the CUDA library for sm_103a into an in-tree shared library.

nvcc compiles each translation unit (one per activation dtype, plus the C-ABI
unit) in parallel, then links ``_build/libfar.so``; g++ compiles the PyTorch
binding of the per-head and block-scaled operators beside them, linked against
it as ``_build/_far_torch.so``.  No GPU is needed: nvcc
cross-compiles.  ``-fmad=false`` keeps every binary32 add and multiply
separately rounded (the kernels also use explicit rounding intrinsics); IEEE
division and square root are nvcc's defaults and are kept (no fast-math).
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libfar.so")
BINDING = os.path.join(BUILD, "_far_torch.so")
BINDING_SOURCE = "far_torch.cpp"
SOURCES = ["far_api.cu", "far_inst_f16.cu", "far_inst_bf16.cu", "far_inst_f32.cu", "far_inst_q_f16.cu",
           "far_inst_q_bf16.cu", "far_inst_q_f32.cu", "far_inst_ln_f16.cu", "far_inst_ln_bf16.cu",
           "far_inst_ln_f32.cu", "far_inst_qb_f16.cu", "far_inst_qb_bf16.cu", "far_inst_qb_f32.cu", "far_noalloc.cu",
           "far_gemm.cu", "far_qk.cu", "far_qblock.cu", "far_gemm8.cu"]
HEADERS = ["far_launch.h", "far_region.h", "far_device.cuh", "far_kernels.cuh", "far_params.h", "far_tcgen05.cuh", "far_tma.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-fmad=false",
                     "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
                     "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _torch_flags() -> tuple[list, list]:
    """g++'s compile and link flags for a Python module on PyTorch's C++ API."""
    import torch

    t = os.path.dirname(torch.__file__)
    lib = os.path.join(t, "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [sysconfig.get_paths()["include"], os.path.join(t, "include"),
           os.path.join(t, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda if os.path.isdir(os.path.join(cuda, "include")) else "/usr/local/cuda", "include"),
           os.path.join(ROOT, "include")]
    cc = ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *(f"-I{i}" for i in inc)]
    ld = ["-shared", f"-L{lib}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{lib}",
          f"-L{BUILD}", "-lfar", "-Wl,-rpath,$ORIGIN"]
    return cc, ld


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + [BINDING_SOURCE]] + [os.path.join(ROOT, "include", "far.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    cc, ld = _torch_flags()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        if src == BINDING_SOURCE:
            cmd = ["g++", *cc, "-c", os.path.join(CSRC, src), "-o", obj]
        else:
            cmd = [nvcc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        *results, (binding, _) = ex.map(compile_one, SOURCES + [BINDING_SOURCE])
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for (_, log), src in zip(results, SOURCES):
            f.write(f"==== {src}\n{log}\n")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = BINDING + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", binding, "-o", tmp, *ld], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)

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
BINDING_STAMP = os.path.join(BUILD, "_far_torch.built_for")  # the Python and PyTorch that the binding was built for
SOURCES = ["far_api.cu", "far_inst_f16.cu", "far_inst_bf16.cu", "far_inst_f32.cu", "far_inst_q_f16.cu",
           "far_inst_q_bf16.cu", "far_inst_q_f32.cu", "far_inst_ln_f16.cu", "far_inst_ln_bf16.cu",
           "far_inst_ln_f32.cu", "far_inst_qb_f16.cu", "far_inst_qb_bf16.cu", "far_inst_qb_f32.cu", "far_noalloc.cu",
           "far_gemm.cu", "far_qk.cu", "far_qblock.cu", "far_gemm8.cu", "far_int8.cu", "far_ffn.cu"]
HEADERS = ["far_launch.h", "far_region.h", "far_device.cuh", "far_kernels.cuh", "far_params.h", "far_tcgen05.cuh", "far_tma.h", "far_pair16.cuh"]
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


def _built_for() -> str:
    import torch

    return f"python {sys.version.split()[0]}, torch {torch.__version__} at {os.path.dirname(torch.__file__)}\n"


def _older(target: str, sources: list) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in sources)


def _library_stale() -> bool:
    return _older(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(ROOT, "include", "far.h")])


def _binding_stale() -> bool:
    """Older than its sources, or built for another Python or PyTorch (whose symbols it would miss)."""
    if _older(BINDING, [os.path.join(CSRC, BINDING_SOURCE), os.path.join(ROOT, "include", "far.h")]):
        return True
    if not os.path.exists(BINDING_STAMP):
        return True
    with open(BINDING_STAMP) as f:
        return f.read() != _built_for()


def _stale() -> bool:
    return _library_stale() or _binding_stale()


def build(force: bool = False, verbose: bool = False) -> str:
    library, binding = force or _library_stale(), force or _binding_stale()
    if not (library or binding):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    cc, ld = _torch_flags() if binding else ([], [])

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
        return r.stderr

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        compiler = ["g++", *cc] if src == BINDING_SOURCE else [nvcc, *NVCC_FLAGS]
        return obj, run([*compiler, "-c", os.path.join(CSRC, src), "-o", obj], f"{compiler[0]} failed for {src}")

    def link(cmd, target):
        tmp = target + f".tmp{os.getpid()}"
        run([*cmd, "-o", tmp], "link failed")
        os.replace(tmp, target)

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        module = ex.submit(compile_one, BINDING_SOURCE) if binding else None
        results = list(ex.map(compile_one, SOURCES)) if library else []
    if library:  # first: it does not need the binding
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            for (_, log), src in zip(results, SOURCES):
                f.write(f"==== {src}\n{log}\n")
        link([nvcc, *ARCH, "-shared", *[o for o, _ in results]], LIB)
    if module:
        link(["g++", module.result()[0], *ld], BINDING)
        with open(BINDING_STAMP, "w") as f:
            f.write(_built_for())
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)

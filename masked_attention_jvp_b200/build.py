"""Builds libcausaljvp.so in-tree with nvcc for sm_100a, and the Python extension
_block.so over it with the host compiler.

Run as `python -m masked_attention_jvp_b200.build` (or call `build()`). The
library is written next to this file so it travels with the source tree; no
JIT cache is involved.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libcausaljvp.so")
SOURCES = ["api.cpp", "api_block.cpp", "api_linear.cpp", "fwd_jvp_sm100.cu", "fwd_jvp_simt.cu", "prologue.cu", "bwd_sm100.cu",
           "host_static.cu", "signal.cu", "out_proj_sm100.cu",
           "qk_rope.cu", "ckpt8.cu", "linear_sm100.cu"]
HEADERS = ["api_internal.h", "kernels.h", "mask_schedule.h", "ptx_sm100.cuh", "vec8.cuh", "ckpt8.cuh",
           "linear_act.cuh", "pair_sm100.cuh", "launch.h"]

# Python entry of the block operators (torch tensors in, the library's calls below)
BIND = "bind.cpp"
EXT = os.path.join(PKG, "_block.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-Xptxas", "-v", "-diag-suppress", "177"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(EXT)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + [BIND]] + [os.path.join(INCLUDE, "causaljvp.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def _build_ext() -> None:
    """_block.so: a CPython extension against this interpreter's torch, linked to the library
    beside it."""
    import sysconfig

    import torch

    torch_dir = os.path.dirname(torch.__file__)
    torch_lib, torch_inc = os.path.join(torch_dir, "lib"), os.path.join(torch_dir, "include")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    incs = [INCLUDE, torch_inc, os.path.join(torch_inc, "torch", "csrc", "api", "include"), sysconfig.get_path("include"), cuda_inc]
    tmp = EXT + f".tmp{os.getpid()}"
    # the system's g++, as nvcc uses: a compiler that links its own static libstdc++ would put
    # a second, uninitialised C++ runtime beside torch's, and the first formatted error crashes
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for i in incs:
        cmd += ["-isystem", i]
    cmd += [os.path.join(CSRC, BIND), "-o", tmp, LIB, f"-L{torch_lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building _block.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = [os.path.join(objdir, src + ".o") for src in SOURCES]

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd.insert(1, "-x")
            cmd.insert(2, "cu")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
        logs = list(pool.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static", "-Xlinker",
                        "-soname=libcausaljvp.so"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _build_ext()
    with open(os.path.join(objdir, "ptxas.log"), "w") as f:
        f.write("\n".join(logs))
    if verbose:
        print("\n".join(logs))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)

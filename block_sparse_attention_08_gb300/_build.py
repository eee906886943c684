"""Builds libmsa.so (the CUDA kernels and the C ABI) for sm_103a with nvcc, and
the extension module that calls it for the chunked-serving functions with g++.

Both are built in-tree under ``_build/`` so the process that loads them loads
them from the repository.  Translation units compile in parallel.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmsa.so")
SOURCES = ["abi.cu", "decode_select.cu", "sparse_attend.cu", "prefill_select.cu", "prefill_attend.cu", "pack.cu",
           "diag.cu", "index_produce.cu", "map_slots.cu", "rotary.cu", "chunk_attend.cu"]
EXT_SOURCE = "serving_ext.cpp"
EXT = os.path.join(BUILD, f"msa_serving-{torch.__version__}.so")  # of this PyTorch
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmsa")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "msa.h"))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(EXT):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)
        return obj

    home = os.path.dirname(torch.__file__)

    def compile_ext():
        obj = os.path.join(BUILD, EXT_SOURCE.replace(".cpp", ".o"))
        include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
                   sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in include),
               "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {EXT_SOURCE}:\n{r.stdout}\n{r.stderr}")
        return obj

    def link(cmd, to):
        tmp = to + f".tmp{os.getpid()}"
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, to)

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(compile_ext)
        objs = list(ex.map(compile_one, SOURCES))
    link([nvcc, *ARCH, "-shared", *objs], LIB)
    # the extension finds libmsa beside itself, and PyTorch's libraries where the process has loaded them
    link(["g++", "-shared", ext.result(), f"-L{BUILD}", "-l:libmsa.so", "-Wl,-rpath,$ORIGIN",
          f"-L{os.path.join(home, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
          "-lc10_cuda"], EXT)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))

"""Builds libmsa.so (the CUDA kernels and the C ABI) for sm_103a with nvcc, and,
for the calls that go through it, the extension module of the chunked-serving
functions with g++.

Both are built in-tree under ``_build/`` so the process that loads them loads
them from the repository.  Translation units compile in parallel.  The module
needs what libmsa does not (g++, Python's headers, a PyTorch with CUDA), so it
is built and loaded only where one of its functions is called.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmsa.so")
SOURCES = ["abi.cu", "decode_select.cu", "sparse_attend.cu", "prefill_select.cu", "prefill_attend.cu", "pack.cu",
           "diag.cu", "index_produce.cu", "map_slots.cu", "rotary.cu", "chunk_attend.cu", "quantize.cu"]
EXT_SOURCE = "serving_ext.cpp"
GXX = "g++"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmsa")


def ext_path() -> str:
    """The extension module of this PyTorch and this Python (it uses the whole interface of both)."""
    import torch
    return os.path.join(BUILD, f"msa_serving-{torch.__version__}-{sysconfig.get_config_var('SOABI')}.so")


def _stale(built, files) -> bool:
    return not os.path.exists(built) or any(os.path.getmtime(f) > os.path.getmtime(built) for f in files)


def _header():
    return os.path.join(INCLUDE, "msa.h")


def up_to_date() -> bool:
    """Whether libmsa is."""
    return not _stale(LIB, [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != EXT_SOURCE] + [_header()])


def _run(cmd, what):
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{what}: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _link(cmd, to):
    tmp = to + f".tmp{os.getpid()}"
    _run([*cmd, "-o", tmp], "link failed")
    os.replace(tmp, to)


def _compile_ext() -> str:
    import torch
    home = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, EXT_SOURCE.replace(".cpp", ".o"))
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    _run([GXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in include),
          "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj], f"{GXX} failed on {EXT_SOURCE}")
    return obj


def build(force: bool = False, verbose: bool = False, serving: bool = False) -> str:
    """Builds what is missing or stale of libmsa and, with ``serving``, of the extension module."""
    lib = force or not up_to_date()
    ext = serving and (force or _stale(ext_path(), [os.path.join(CSRC, EXT_SOURCE), _header()]))
    if not lib and not ext:
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        out = _run([_nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj], f"nvcc failed on {src}")
        if verbose:
            print(out)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext_obj = ex.submit(_compile_ext) if ext else None
        if lib:
            _link([_nvcc(), *ARCH, "-shared", *ex.map(compile_one, SOURCES)], LIB)
        if ext:
            import torch
            # the module finds libmsa beside itself, and PyTorch's libraries where the process has loaded them
            _link([GXX, "-shared", ext_obj.result(), f"-L{BUILD}", "-l:libmsa.so", "-Wl,-rpath,$ORIGIN",
                   f"-L{os.path.join(os.path.dirname(torch.__file__), 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
                   "-ltorch_cuda", "-lc10", "-lc10_cuda"], ext_path())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True, serving=True))

"""Build libdecode_attn.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ compiles to an object in parallel, then one nvcc call
links the shared library (static CUDA runtime, no libcuda link: the TMA
encoder is fetched through the runtime's driver entry-point query).  The
CPython extension native/calls.cpp (host code, against torch's headers) builds
at the same time into lib/_calls.so, which finds the library beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libdecode_attn.so")
CALLS_SRC = os.path.join(PKG, "native", "calls.cpp")
CALLS_PATH = os.path.join(LIB_DIR, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    cand = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cand, "bin", "nvcc")
    return path if os.path.exists(path) else (shutil.which("nvcc") or "nvcc")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                        if f.endswith((".cuh", ".h"))] + \
        [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _compile(src: str, verbose_ptxas: bool, extra=(), build_dir=BUILD_DIR) -> str:
    obj = os.path.join(build_dir, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd[1:1] = ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas and res.stderr:
        print(res.stderr)
    return obj


def _compile_calls(obj: str) -> str:
    """Compile native/calls.cpp; returns torch's library folder."""
    import torch
    torch_inc = os.path.join(os.path.dirname(torch.__file__), "include")
    incs = [INCLUDE, sysconfig.get_paths()["include"], torch_inc,
            os.path.join(torch_inc, "torch", "csrc", "api", "include"),
            os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(x for i in incs for x in ("-isystem" if i != INCLUDE else "-I", i)), "-c", CALLS_SRC,
           "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALLS_SRC}:\n{res.stdout}\n{res.stderr}")
    return os.path.join(os.path.dirname(torch.__file__), "lib")


def _link_calls(obj: str, torch_lib: str) -> None:
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", torch_lib, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L", LIB_DIR, "-ldecode_attn", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking _calls.so failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, CALLS_PATH)


def _fresh(path: str, deps) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(d) for d in deps)


def build(force: bool = False, verbose_ptxas: bool = False, extra_flags=(),
          lib_path: str = LIB_PATH) -> str:
    """Compile csrc/*.cu and link lib/libdecode_attn.so (or `lib_path`, with
    `extra_flags` such as -D overrides of the pipeline shape); returns its path."""
    own = lib_path == LIB_PATH  # (an overridden library has no extension beside it)
    build_dir = BUILD_DIR if own else os.path.dirname(lib_path) + "/_obj"
    os.makedirs(build_dir, exist_ok=True)
    os.makedirs(os.path.dirname(lib_path), exist_ok=True)
    calls_deps = [CALLS_SRC, os.path.join(INCLUDE, "decode_attn.h")]
    need_lib = force or not _fresh(lib_path, _deps())
    need_calls = own and (force or not _fresh(CALLS_PATH, calls_deps))
    if not need_lib and not need_calls:
        return lib_path
    srcs = sources() if need_lib else []
    obj = os.path.join(build_dir, "calls.o")
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        calls = ex.submit(_compile_calls, obj) if need_calls else None
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas, tuple(extra_flags), build_dir),
                           srcs))
    if need_lib:
        tmp = lib_path + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, lib_path)
    if calls is not None:
        _link_calls(obj, calls.result())
    return lib_path


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose_ptxas="-v" in sys.argv))

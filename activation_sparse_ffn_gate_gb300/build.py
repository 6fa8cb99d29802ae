"""Build libtwell_gb300.so in-tree with nvcc for sm_103a, and the native calls (_twell_call.so) with g++.

Each CUDA translation unit is compiled in parallel, then linked into one shared library with the
static CUDA runtime (no link-time dependency on libcuda: the TMA descriptor encoder is fetched
from the driver at run time). The native calls are one C++ file against PyTorch's headers, linked to that library.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtwell_gb300.so")
CALL = os.path.join(PKG, "_twell_call.so")
STAMP = os.path.join(BUILD, "twell_call.stamp")

SOURCES = ["twell_host.cu", "twell_gate.cu", "twell_ffn.cu", "twell_pack.cu", "twell_hybrid.cu", "twell_light.cu",
           "twell_union.cu", "twell_union_small.cu", "twell_decode.cu", "twell_tile_union.cu", "twell_norm.cu",
           "twell_kv.cu", "twell_attn.cu", "twell_w4.cu", "twell_rope.cu", "twell_plan.cu", "twell_lora.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr",
              "-I" + INCLUDE, "-I" + CSRC]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "twell.h")]
    return max(os.path.getmtime(f) for f in files)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")


def _call_flags():
    """Compiler and linker flags of the native calls: PyTorch's headers and libraries, CUDA's headers, Python's."""
    import sysconfig

    import torch
    torch_dir = os.path.dirname(torch.__file__)
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    lib = os.path.join(torch_dir, "lib")
    compile_flags = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I" + INCLUDE,
                     f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in inc:
        compile_flags += ["-isystem", d]
    link_flags = ["-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath," + lib, "-L" + PKG,
                  "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    return compile_flags, link_flags


def _call_stamp():
    """What the native calls were built for besides their sources: PyTorch and Python."""
    import torch
    return f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, python {sys.version}\n"


def _stale():
    """Whether the library, and whether the native calls beside it, have to be built."""
    def old(f):
        return not os.path.exists(f) or os.path.getmtime(f) < _deps()

    lib = old(LIB)
    if lib or old(CALL) or not os.path.exists(STAMP):
        return lib, True
    with open(STAMP) as f:
        return lib, f.read() != _call_stamp()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    lib_stale, call_stale = (True, True) if force else _stale()
    if not call_stale:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        return obj

    compile_flags, link_flags = _call_flags()

    def compile_call():
        obj = os.path.join(BUILD, "twell_call.o")
        _run(["g++", *compile_flags, "-c", os.path.join(CSRC, "twell_call.cpp"), "-o", obj], "g++ failed for twell_call.cpp")
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        call_obj = ex.submit(compile_call)
        if lib_stale:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + f".{os.getpid()}.tmp"
            cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
            _run(cmd, "link failed")
            os.replace(tmp, LIB)
        call_obj = call_obj.result()  # the library is there by now: its own calls run without these
    tmp = CALL + f".{os.getpid()}.tmp"
    _run(["g++", "-shared", "-o", tmp, call_obj, *link_flags], "link of the native calls failed")
    os.replace(tmp, CALL)
    with open(STAMP, "w") as f:
        f.write(_call_stamp())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))

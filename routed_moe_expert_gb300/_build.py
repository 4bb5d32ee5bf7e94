"""Build the in-tree shared library libmoelora.so (sm_103a) with nvcc, and the Python module
_marshal.so (argument marshalling against PyTorch's C++ interface) with g++.

Each .cu file is compiled in parallel to an object under _build/, then linked into
routed_moe_expert_gb300/libmoelora.so with the CUDA runtime linked statically, so the
library needs no CUDA shared object at load time (the driver is loaded lazily on the
first CUDA call).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoelora.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_ABI = os.path.join(PKG, "_marshal.abi")   # what the module beside it was built against
SOURCES = ["moe_lora.cu", "route_align.cu", "grouped_gemm.cu", "gemm_fp8.cu", "elementwise.cu", "lora.cu", "route_noalloc.cu",
           "lora_tc.cu", "permute_shrink.cu", "nvfp4.cu", "select_experts.cu", "qk_norm_rope.cu",
           "page_cache.cu", "attention.cu", "attention_rows.cu", "attention_tiles.cu", "linear.cu", "linear_narrow.cu", "linear_wide.cu", "linear_cluster.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoelora.so")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "moe_lora.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def marshal_abi() -> str:
    """What _marshal.so depends on besides its sources: this Python and this PyTorch."""
    import torch
    return f"Python {sys.version_info[0]}.{sys.version_info[1]}, PyTorch {torch.__version__}"


def marshal_built_for() -> str:
    """What the _marshal.so in place was built against ("" when that is not known)."""
    try:
        with open(MARSHAL_ABI) as f:
            return f.read()
    except OSError:
        return ""


def _build_marshal(verbose: bool) -> None:
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    lib = os.path.join(base, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", os.path.join(CSRC, "binding.cpp"), "-o", MARSHAL + ".tmp"]
    for d in inc:
        cmd += ["-isystem", d]
    cmd += [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-L", lib, f"-Wl,-rpath,{lib}",
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    if verbose:
        print(r.stdout + r.stderr)
    if os.path.exists(MARSHAL_ABI):
        os.remove(MARSHAL_ABI)
    os.replace(MARSHAL + ".tmp", MARSHAL)
    with open(MARSHAL_ABI, "w") as f:
        f.write(marshal_abi())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libmoelora.so if any source is newer than it, and _marshal.so if any is or it was
    built against another Python or PyTorch.  The library does not depend on the module: it is in
    place also when building the module fails, which raises.  Returns the library's path."""
    fresh = {f: not force and os.path.exists(f) and os.path.getmtime(f) >= _deps_mtime() for f in (LIB, MARSHAL)}
    fresh[MARSHAL] = fresh[MARSHAL] and marshal_built_for() == marshal_abi()
    if all(fresh.values()):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        marshal = None if fresh[MARSHAL] else ex.submit(_build_marshal, verbose)
        if not fresh[LIB]:
            _build_library(verbose)
        if marshal is not None:
            marshal.result()
    return LIB


def _build_library(verbose: bool) -> None:
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

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force=True, verbose=True))

"""Build libklt.so (the C-ABI tail library) in-tree with nvcc for sm_103a.

Each .cu file compiles to an object in parallel, then one shared-library link.  The
library links the CUDA runtime dynamically and reaches the driver's tensor-map encoder
through the runtime's entry-point query, so it loads on a machine without a GPU driver
(its entry points then fail with a CUDA status instead of refusing to load).  A small CPython
module beside it marshals the arguments of the operators around the tail.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
OUT_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libklt.so")
MARSHAL_PATH = os.path.join(PKG_DIR, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["klt_api.cu", "klt_route.cu", "klt_gemm.cu", "klt_wide.cu", "klt_noalloc.cu",
           "klt_block.cu", "klt_linear.cu", "klt_linear_narrow.cu", "klt_linear_wide.cu"]
HEADERS = ["klt_device.cuh", "klt_internal.h", "klt_linear.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False, ptxas_info: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "klt.h")]

    def compile_one(src: str) -> str:
        path = os.path.join(CSRC, src)
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        if force or _stale(obj, [path] + hdrs):
            cmd = [nvcc, *ARCH, *FLAGS, "-c", path, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
            if verbose or ptxas_info:
                sys.stderr.write(res.stdout + res.stderr)
        return obj

    # the CPython module of the operators' calls, against torch's headers
    gxx = shutil.which("g++") or "g++"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]

    def compile_marshal() -> str:
        path, obj = os.path.join(CSRC, "klt_marshal.cpp"), os.path.join(OUT_DIR, "klt_marshal.o")
        if force or _stale(obj, [path, hdrs[-1], os.path.join(torch_dir, "version.py")]):
            cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-Wall", "-c", path, "-o", obj]
            cmd += ["-I" + d for d in (os.path.join(torch_dir, "include"),
                                       os.path.join(cuda, "include"),
                                       sysconfig.get_paths()["include"])]
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"g++ failed for klt_marshal.cpp:\n{res.stdout}\n{res.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(compile_marshal)
        objs = list(ex.map(compile_one, SOURCES))
        marshal_obj = marshal.result()
    if force or _stale(LIB_PATH, objs):
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", LIB_PATH, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    if force or _stale(MARSHAL_PATH, [marshal_obj, LIB_PATH]):
        cmd = [gxx, "-shared", marshal_obj, "-o", MARSHAL_PATH, "-L" + PKG_DIR, "-l:libklt.so",
               "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
               "-lc10_cuda", "-L" + os.path.join(cuda, "lib64"), "-lcudart",
               "-Wl,-rpath,$ORIGIN:" + os.path.join(torch_dir, "lib")]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed for _marshal:\n{res.stdout}\n{res.stderr}")
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv, ptxas_info="-v" in sys.argv))

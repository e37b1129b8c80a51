"""Build libklt.so (the C-ABI tail library) in-tree with nvcc for sm_103a.

Each .cu file compiles to an object in parallel, then one shared-library link.  The
library links the CUDA runtime dynamically and reaches the driver's tensor-map encoder
through the runtime's entry-point query, so it loads on a machine without a GPU driver
(its entry points then fail with a CUDA status instead of refusing to load).  A small CPython
module beside it marshals the arguments of the operators around the tail; the library and the tail
need neither it nor torch's headers.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
OUT_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libklt.so")
EXT_SUFFIX = sysconfig.get_config_var("EXT_SUFFIX")  # names the interpreter and the machine
MARSHAL_PATH = os.path.join(PKG_DIR, "_marshal" + EXT_SUFFIX)
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


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise ImportError("torch is not installed")
    return spec.submodule_search_locations[0]


def _gxx(cmd, what: str) -> None:
    res = subprocess.run([shutil.which("g++") or "g++", *cmd], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {what}:\n{res.stdout}\n{res.stderr}")


def _cuda_dir(nvcc: str) -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))


def _compile_marshal(nvcc: str, header: str, force: bool) -> str:
    """The CPython module of the operators' calls, against torch's and this interpreter's
    headers."""
    torch_dir = _torch_dir()
    path = os.path.join(CSRC, "klt_marshal.cpp")
    obj = os.path.join(OUT_DIR, "klt_marshal" + EXT_SUFFIX + ".o")
    if force or _stale(obj, [path, header, os.path.join(torch_dir, "version.py")]):
        import torch
        includes = (os.path.join(torch_dir, "include"), os.path.join(_cuda_dir(nvcc), "include"),
                    sysconfig.get_paths()["include"])
        _gxx(["-O2", "-std=c++17", "-fPIC", "-Wall",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
              *("-I" + d for d in includes), "-c", path, "-o", obj], "klt_marshal.cpp")
    return obj


def _link_marshal(nvcc: str, obj: str, force: bool) -> None:
    if not force and not _stale(MARSHAL_PATH, [obj, LIB_PATH]):
        return
    torch_lib = os.path.join(_torch_dir(), "lib")
    _gxx(["-shared", obj, "-o", MARSHAL_PATH, "-L" + os.path.dirname(LIB_PATH), "-l:libklt.so",
          "-L" + torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
          "-L" + os.path.join(_cuda_dir(nvcc), "lib64"), "-lcudart",
          "-Wl,-rpath,$ORIGIN:" + torch_lib], "_marshal")


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

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(_compile_marshal, nvcc, hdrs[-1], force)
        objs = list(ex.map(compile_one, SOURCES))
    if force or _stale(LIB_PATH, objs):
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", LIB_PATH, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    try:
        _link_marshal(nvcc, marshal.result(), force)
    except (RuntimeError, ImportError, OSError) as e:
        # the library is complete; the operators' Python calls say that their module is missing
        if os.path.exists(MARSHAL_PATH):
            os.remove(MARSHAL_PATH)
        warnings.warn(f"the operators' Python module is not built: {e}", RuntimeWarning)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv, ptxas_info="-v" in sys.argv))

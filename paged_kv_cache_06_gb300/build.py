"""Build libpagedkv.so in-tree from csrc/ (nvcc for sm_103a, g++ for host code),
and the Python binding of the drafted step's calls, ``_binding.so``.

Translation units compile in parallel into ``_build/`` and link into
``paged_kv_cache_06_gb300/libpagedkv.so``; ``csrc/python/`` compiles against the
installed torch's headers into ``_binding.so`` beside it, which links to it.
Rebuilds only when a source or header is newer than the products.  Usage: ``python -m
paged_kv_cache_06_gb300.build [--force]``.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libpagedkv.so")
BINDING_SRC = os.path.join(CSRC, "python", "binding.cpp")
BINDING_PATH = os.path.join(HERE, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.isdir(home):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _nvcc() -> str:
    return os.path.join(_cuda_home(), "bin", "nvcc")


def sources():
    cu = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    cpp = sorted(glob.glob(os.path.join(CSRC, "*.cpp")))
    return cu, cpp


def _inputs():
    cu, cpp = sources()
    hdr = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return cu + cpp + hdr + [BINDING_SRC]


def is_stale() -> bool:
    if not (os.path.exists(LIB_PATH) and os.path.exists(BINDING_PATH)):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return any(os.path.getmtime(p) > t for p in _inputs())


def _torch_dir() -> str:
    """The installed torch's folder, without importing it."""
    import importlib.util
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _binding_flags():
    torch_inc = os.path.join(_torch_dir(), "include")
    return ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE,
            "-isystem", torch_inc, "-isystem", os.path.join(torch_inc, "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(_cuda_home(), "include"),
            "-isystem", sysconfig.get_config_var("INCLUDEPY")]


def _compile(src: str, verbose: bool, ptxas_info: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cuda_inc = os.path.join(_cuda_home(), "include")
    if src == BINDING_SRC:
        cmd = [os.environ.get("CXX", "g++"), *_binding_flags(), "-c", src, "-o", obj]
    elif src.endswith(".cu"):
        cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
               "-I", INCLUDE, "-c", src, "-o", obj]
        if ptxas_info:
            cmd[1:1] = ["-Xptxas", "-v"]
    else:
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wall",
               "-I", INCLUDE, "-I", cuda_inc, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0 or ptxas_info:
        sys.stderr.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"compiling {os.path.basename(src)} failed:\n{res.stderr}")
    return obj


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every CUDA/C++ source for sm_103a and link libpagedkv.so."""
    if not force and not ptxas_info and not is_stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cu, cpp = sources()
    srcs = [BINDING_SRC] + cu + cpp  # the slowest first
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        binding, *objs = ex.map(lambda s: _compile(s, verbose, ptxas_info), srcs)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    lib_dir = os.path.join(_cuda_home(), "lib64")
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-L", lib_dir, "-Xlinker", f"-rpath,{lib_dir}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking libpagedkv.so failed:\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    torch_lib = os.path.join(_torch_dir(), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, binding, "-L", HERE, "-l:libpagedkv.so",
           "-Wl,-rpath,$ORIGIN", "-L", torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-L", lib_dir, "-lcudart", f"-Wl,-rpath,{torch_lib}", f"-Wl,-rpath,{lib_dir}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking _binding.so failed:\n{res.stderr}")
    os.replace(tmp, BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv,
          ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)

"""Build libpagedkv.so in-tree from csrc/ (nvcc for sm_103a, g++ for host code),
and the Python binding of the drafted step's calls, ``_binding.so``.

Translation units compile in parallel into ``_build/`` and link into
``paged_kv_cache_06_gb300/libpagedkv.so``, for which nvcc and g++ are enough;
``csrc/python/`` compiles against the installed torch's and Python's headers into
``_binding.so`` beside it, which links to it, and is left out where there is no
torch.  Rebuilds only when a source or header is newer than the product, and the
binding also when torch or Python is another one.  Usage: ``python -m
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


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _older(product: str, inputs) -> bool:
    return not os.path.exists(product) or any(os.path.getmtime(p) > os.path.getmtime(product) for p in inputs)


def library_is_stale() -> bool:
    cu, cpp = sources()
    return _older(LIB_PATH, cu + cpp + _headers())


def _torch_dir() -> str | None:
    """The installed torch's folder, without importing it (None: no torch)."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _binding_stamp() -> str:
    """What the binding was compiled against."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return "\n".join([sys.version, str(sysconfig.get_config_var("SOABI")), _torch_dir(), f.read()])


def binding_is_stale() -> bool:
    if _older(BINDING_PATH, _headers() + [BINDING_SRC]):
        return True
    try:
        with open(_stamp_path()) as f:
            return f.read() != _binding_stamp()
    except OSError:
        return True


def _stamp_path() -> str:
    return os.path.join(BUILD_DIR, "binding.stamp")


def is_stale() -> bool:
    return library_is_stale() or (_torch_dir() is not None and binding_is_stale())


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


def _compile_all(srcs, verbose: bool, ptxas_info: bool):
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        return [ex.submit(_compile, s, verbose, ptxas_info) for s in srcs]


def _link(cmd, path: str) -> None:
    tmp = path + f".tmp{os.getpid()}"
    res = subprocess.run([x if x is not None else tmp for x in cmd], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking {os.path.basename(path)} failed:\n{res.stderr}")
    os.replace(tmp, path)


def _link_library(objs) -> None:
    lib_dir = os.path.join(_cuda_home(), "lib64")
    _link([_nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", None, *objs,
           "-L", lib_dir, "-Xlinker", f"-rpath,{lib_dir}"], LIB_PATH)


def _link_binding(obj: str) -> None:
    lib_dir = os.path.join(_cuda_home(), "lib64")
    torch_lib = os.path.join(_torch_dir(), "lib")
    _link([os.environ.get("CXX", "g++"), "-shared", "-o", None, obj, "-L", HERE, "-l:libpagedkv.so",
           "-Wl,-rpath,$ORIGIN", "-L", torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-L", lib_dir, "-lcudart", f"-Wl,-rpath,{torch_lib}", f"-Wl,-rpath,{lib_dir}"],
          BINDING_PATH)
    with open(_stamp_path(), "w") as f:
        f.write(_binding_stamp())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False, library: bool = True,
          binding: bool = True) -> str:
    """Compile every CUDA/C++ source for sm_103a and link libpagedkv.so, then the
    binding (where torch is installed); either may be left out.  The library does not
    depend on the binding: it is linked before the binding's errors are raised."""
    library = library and (force or ptxas_info or library_is_stale())
    binding = binding and _torch_dir() is not None and (force or binding_is_stale())
    cu, cpp = sources()
    # the slowest first
    srcs = ([BINDING_SRC] if binding else []) + (cu + cpp if library else [])
    if not srcs:
        return LIB_PATH
    objs = _compile_all(srcs, verbose, ptxas_info)
    if library:
        _link_library([o.result() for o in objs[binding:]])
    if binding:
        _link_binding(objs[0].result())
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv,
          ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)

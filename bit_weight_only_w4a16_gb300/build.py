"""Build libw4a16.so in-tree with nvcc for sm_103a (no cmake; parallel objects), and the
serving calls' native binding with g++ against the installed torch."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libw4a16.so")
BUILD_DIR = os.path.join(os.path.dirname(HERE), "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    n = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(n):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libw4a16.so")
    return n


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def binding_path() -> str:
    """The native binding for this torch and this Python: it uses the layout of their objects, so one that
    was built for others has another name and is neither current nor loaded."""
    import torch
    git = (torch.version.git_version or "")[:10]
    return os.path.join(HERE, f"_binding.{torch.__version__}.{git}{sysconfig.get_config_var('EXT_SUFFIX')}")


def binding_current() -> bool:
    path = binding_path()
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in
                                        (os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "w4a16.h")))


def build_binding(force: bool = False):
    """The native binding's path, or None where it cannot be built (the Python binding is
    complete without it; only the host time of the serving calls is longer)."""
    try:
        import torch
        if not force and binding_current():
            return binding_path()
        src, path = os.path.join(CSRC, "binding.cpp"), binding_path()
        base = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(_nvcc()))
        tmp = path + ".tmp"
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", src, "-o", tmp, "-I", os.path.join(base, "include"),
               "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"), "-I",
               sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-L", os.path.join(base, "lib"),
               "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(r.stderr[-2000:])
        os.replace(tmp, path)
        return path
    except Exception as e:  # noqa: BLE001
        print(f"the native binding was not built: {e}", file=sys.stderr)
        return None


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        build_binding()
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = extra or []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(2, min(8, os.cpu_count() or 2))) as ex:
        binding = ex.submit(build_binding, force)
        objs = list(ex.map(compile_one, _sources()))
        binding.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))

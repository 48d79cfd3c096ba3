"""Build the CUDA library libmoe_decode.so in-tree with nvcc (sm_103a only).

Each .cu file under csrc/ is compiled to an object in parallel, then linked
into one shared library next to this file. The CUDA runtime is linked
statically, so the library needs only the driver at run time. A second, small
module (torch_calls.cpp) takes torch tensors to the operators' entry points; it
is built where torch is installed, for that version of it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libmoe_decode.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
# translation units whose kernels move registers between warpgroups (setmaxnreg)
SPLIT_SOURCES = ("decode_step.cu",)
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
          "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _cuda_include() -> str:
    """The CUDA headers: nvcc's, or where the toolkit usually is."""
    try:
        home = os.path.dirname(os.path.dirname(_nvcc()))
    except RuntimeError:
        home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return os.path.join(home, "include")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def calls_path():
    """Where the torch_calls module for this interpreter and the installed torch is built
    (it is tied to both); None without a torch that has CUDA."""
    try:
        import torch
    except (ImportError, OSError):
        return None
    if torch.version.cuda is None:
        return None
    version = "".join(c if c.isalnum() else "_" for c in torch.__version__)
    return os.path.join(PKG, f"_torch_calls_{version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_calls(force: bool = False):
    """Compile torch_calls.cpp with the host compiler; returns its path, or None where that
    is not possible (no C++ compiler, no Python headers): calls then go through ctypes."""
    path = calls_path()
    if path is None:
        return None
    src = os.path.join(CSRC, "torch_calls.cpp")
    deps = [src, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps):
        return path
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [INCLUDE, os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], _cuda_include()]
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", *[f"-I{d}" for d in inc],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", src, "-o", tmp,
           "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = r.returncode and f"{cmd[0]} failed:\n{r.stdout}\n{r.stderr}"
    except OSError as e:
        why = str(e)
    if why:
        if os.path.exists(path):  # of older sources
            os.remove(path)
        warnings.warn(f"{src} is not built, calls of the operators go through ctypes: {why}")
        return None
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link; returns the library path. Skips work when up to date."""
    if not force and up_to_date():
        build_calls()
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = ARCH_FLAGS + COMMON + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src).replace(".cu", ".o"))
        split = os.path.basename(src) in SPLIT_SOURCES
        cmd = [nvcc, *flags, *(["-Xptxas", "-v"] if split else []), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if split and "setmaxnreg' ignored" in r.stdout + r.stderr:
            # the kernel would run, but every warp would keep the launch's
            # register count instead of the consumer / producer split
            raise RuntimeError(f"ptxas dropped the setmaxnreg register split of {src}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        calls = ex.submit(build_calls, force)
        objs = list(ex.map(compile_one, srcs))
        calls.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))

"""In-tree build of libint8conv.so (nvcc, sm_103a only) and of the channel
operators' Python binding.

Every translation unit under ``csrc/`` is compiled in parallel into
``_build/`` and linked into ``libint8conv.so`` next to this file;
``csrc/python/channel_binding.cpp`` is compiled against torch's headers into
``_channel.so``, which loads the library.  Rebuilds only what is older than a
source or header, and the binding where it was built for another Python or
torch; without torch the library alone is built (its C entry points need none).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libint8conv.so")
BINDING_SRC = os.path.join(CSRC, "python", "channel_binding.cpp")
BINDING = os.path.join(PKG, "_channel.so")
BINDING_STAMP = os.path.join(OBJDIR, "channel_binding.txt")  # what the binding was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libint8conv.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def torch_root() -> str | None:
    """Where torch is installed (without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def binding_target() -> str:
    """The Python and the torch that a binding built now would be for."""
    with open(os.path.join(torch_root(), "version.py")) as f:
        return f"{sys.version}\n{sysconfig.get_paths()['include']}\n{torch_root()}\n{f.read()}"


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_STAMP):
        return False
    t = os.path.getmtime(BINDING)
    deps = [BINDING_SRC, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    with open(BINDING_STAMP) as f:
        return all(os.path.getmtime(d) <= t for d in deps) and f.read() == binding_target()


def build_binding() -> None:
    """_channel.so; needs the library next to it to link with."""
    root = torch_root()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-o", tmp, BINDING_SRC, "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
           "-L", PKG, "-l:libint8conv.so", "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(BINDING_SRC)}:\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(OBJDIR, exist_ok=True)
    with open(BINDING_STAMP, "w") as f:
        f.write(binding_target())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    build_library(force, verbose, extra_flags)
    if torch_root() is None:
        print("torch is not installed: the channel operators' Python binding is left out", file=sys.stderr)
    elif force or not binding_up_to_date():
        build_binding()
    return LIB


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        cmd = [cc] + ARCH + FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        if src.endswith(".cpp"):
            cmd = [cc] + FLAGS + list(extra_flags) + ["-x", "c++", "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))

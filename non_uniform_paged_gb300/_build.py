"""Build libtg.so in-tree with nvcc for sm_103a (no CMake, no torch extension).

Each translation unit compiles in its own nvcc process, in parallel; objects
go to ``_build/`` at the repository root and the shared library next to this
file.  The host code is portable C++17 (it builds the same on x86_64 and
aarch64); the device code targets sm_103a only.  Apart from it, g++ builds the Python module _calls
(binding/calls.cpp), which checks torch tensors for the calls whose host time counts: libtg needs
neither torch nor that module.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import hashlib
import os
import re
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libtg.so")
CALLS_SRC = os.path.join(PKG, "binding", "calls.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O3", "-I", INCLUDE,
         "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtg.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _newer(path, inputs) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in inputs)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch not found: its headers are required to build _calls")
    return spec.submodule_search_locations[0]


def calls_path() -> str:
    """Where _calls is for this Python and this torch: the module holds the layout of the one's tensors
    and the other's objects, so each pair has a file of its own."""
    where = _torch_dir()
    with open(os.path.join(where, "version.py")) as f:
        version = re.search(r"__version__\s*=\s*['\"]([^'\"]+)", f.read())
    key = f"{version.group(1) if version else 'unknown'}-{hashlib.sha256(where.encode()).hexdigest()[:8]}"
    return os.path.join(PKG, f"_calls-{key}{sysconfig.get_config_var('EXT_SUFFIX')}")


def calls_up_to_date() -> bool:
    return _newer(calls_path(), [CALLS_SRC, os.path.join(INCLUDE, "tg.h"), os.path.abspath(__file__)])


def build_calls(force: bool = False) -> str:
    """Compile the Python module _calls against the torch that will import it; returns its path."""
    torch_dir, path = _torch_dir(), calls_path()
    if not force and calls_up_to_date():
        return path
    tmp = f"{path}.{os.getpid()}.tmp"  # several processes may meet here at their first call
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-I", os.path.join(torch_dir, "include"), "-I", sysconfig.get_paths()["include"], CALLS_SRC, "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-Wl,-rpath," + os.path.join(torch_dir, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on calls.cpp:\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libtg.so; returns its path.  Raises on any compiler error."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build_all(force: bool = False, verbose: bool = False):
    """libtg.so and _calls, side by side; returns both paths."""
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(build_calls, force)
        return build(force, verbose), calls.result()


if __name__ == "__main__":
    import sys
    print(*build_all(force="--force" in sys.argv, verbose=True))

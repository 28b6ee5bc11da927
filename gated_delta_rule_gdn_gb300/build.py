"""Build libgdn_gb300.so in-tree with nvcc for sm_103a (GB300).

Each translation unit under csrc/ compiles to an object in parallel; the
objects link into gated_delta_rule_gdn_gb300/libgdn_gb300.so.  There is no
cmake and no torch extension machinery: the library is plain C ABI.  The
Python extension module csrc/torch_binding.cpp (tensor checks and allocation
for some entry points) compiles beside them with the host compiler against
torch's headers, into gated_delta_rule_gdn_gb300/_native.so.  It fits the
torch and the Python it was built with alone, so a stamp beside the objects
names them, and another torch or Python means another build.

Environment knobs:
  GDN_NVCC          nvcc to use (default: nvcc on PATH, else /usr/local/cuda/bin/nvcc)
  GDN_CXX           host compiler of the extension module (default: g++ on PATH)
  GDN_PTXAS_VERBOSE=1  pass -Xptxas -v (registers, spills, shared memory per kernel)
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn_gb300.so")
NATIVE = os.path.join(PKG, "_native.so")
STAMP = os.path.join(BUILD, "native.stamp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    env = os.environ.get("GDN_NVCC")
    if env:
        return env
    return shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _native_stamp() -> str:
    """What the extension module depends on besides its source: the torch (its version file names the build) and the Python."""
    with open(os.path.join(_torch_dir(), "version.py"), encoding="utf-8") as f:
        return "\n".join([_torch_dir(), f.read(), sys.version, platform.machine()])


def native_current() -> bool:
    """Whether the extension module was built with the torch and the Python that are here."""
    try:
        with open(STAMP, encoding="utf-8") as f:
            return os.path.exists(NATIVE) and f.read() == _native_stamp()
    except OSError:
        return False


def _native_command(out: str) -> list:
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = os.path.join(torch, "include")
    return [os.environ.get("GDN_CXX") or shutil.which("g++") or "c++", "-O1", "-std=c++20", "-fPIC", "-shared",
            "-I", include, "-I", os.path.join(include, "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
            os.path.join(CSRC, "torch_binding.cpp"), "-o", out, "-L", os.path.join(torch, "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cpp"))) + sorted(glob.glob(os.path.join(CSRC, "*.h"))) + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) \
        + sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not native_current():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(NATIVE))
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library if needed; return its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if os.environ.get("GDN_PTXAS_VERBOSE") == "1":
        flags += ["-Xptxas", "-v"]

    def run(cmd, what: str):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or (verbose and r.stderr):
            sys.stderr.write(r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"compilation failed on {what}")

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        run([nvcc] + flags + ["-c", src, "-o", obj], os.path.basename(src))
        return obj

    def compile_native() -> str:
        out = NATIVE + f".tmp{os.getpid()}"
        run(_native_command(out), "torch_binding.cpp")
        return out

    srcs, stamp = _sources(), _native_stamp()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        native = ex.submit(compile_native)
        objs = list(ex.map(compile_one, srcs))
        native = native.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    os.replace(native, NATIVE)
    with open(STAMP + f".tmp{os.getpid()}", "w", encoding="utf-8") as f:
        f.write(stamp)
    os.replace(f.name, STAMP)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))

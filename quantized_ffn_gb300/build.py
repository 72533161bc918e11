"""Build the CUDA library libzffn.so in-tree for sm_103a (no CMake).

Each translation unit under csrc/ is compiled by nvcc in parallel, then linked
into quantized_ffn_gb300/_lib/libzffn.so (CUDA runtime linked statically; the
driver entry point used for TMA descriptors is looked up at run time).  The
Python binding of the 8-bit entry points (csrc/binding.cpp) is compiled by the
host compiler against the installed torch into _lib/_zffn_native.so; where that
fails, build() warns and the library stands alone.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libzffn.so")
NATIVE = os.path.join(OUT_DIR, "_zffn_native.so")   # beside it NATIVE + ".for": what it was made for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hdrs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hdrs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def native_is_for(native: str) -> str:
    """The torch and the Python that this binding was compiled against ("" where nothing says so)."""
    try:
        with open(native + ".for") as f:
            return f.read()
    except OSError:
        return ""


def native_wanted() -> str:
    """The same of this process: a binding for another pair is not loaded, and built again."""
    import torch

    return f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def _native_stale() -> bool:
    try:
        wanted = native_wanted()
    except ImportError:
        return True
    return native_is_for(NATIVE) != wanted or _stale(NATIVE, [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "zffn.h")])


def _native_command():
    """The host compiler's command line for the binding, with the installed torch's paths."""
    import sysconfig

    import torch

    home = os.path.dirname(torch.__file__)
    lib = os.path.join(home, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    inc = [INCLUDE, os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"), cuda,
           sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *["-I" + i for i in inc],
            os.path.join(CSRC, "binding.cpp"), "-L" + lib, "-Wl,-rpath," + lib,
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    hdrs = _deps()
    objs, jobs = [], []
    for src in sources():
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hdrs):
            cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
            jobs.append(cmd)
    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("the compiler failed: " + " ".join(cmd))

    def bind():
        tmp = NATIVE + f".{os.getpid()}.tmp"
        run(_native_command() + ["-o", tmp])
        os.replace(tmp, NATIVE)
        with open(tmp, "w") as f:
            f.write(native_wanted())
        os.replace(tmp, NATIVE + ".for")

    native = force or _native_stale()
    if jobs or native:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs) + native, os.cpu_count() or 4)) as ex:
            bound = ex.submit(bind) if native else None
            for f in [ex.submit(run, cmd) for cmd in jobs]:
                f.result()
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if native and bound.exception() is not None:
        # the library needs nvcc alone: a host without torch's headers, Python's or a
        # CUDA build of torch keeps it (and the calls that do not go through the binding).
        # A module of other sources is not left to be loaded instead.
        if os.path.exists(NATIVE):
            os.remove(NATIVE)
        warnings.warn(f"{NATIVE} was not built, so the 8-bit and sorting functions are missing from Python: "
                      f"{bound.exception()}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))

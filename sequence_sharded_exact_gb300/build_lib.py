"""Builds libringattn.so in-tree: every csrc/*.cu compiled for sm_103a in parallel, then linked; and beside it the
binding's compiled calls (csrc/calls.cpp, against the installed torch).

Usage: python -m sequence_sharded_exact_gb300.build_lib [--force]
The CUDA runtime is linked statically and the driver API is reached through the runtime's entry
point query, so the library loads on machines without a GPU driver (calls then return
RA_ERR_NO_DEVICE).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libringattn.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "calls.cpp"] + [os.path.join(INCLUDE, "ringattn.h"),
                                                              os.path.abspath(__file__)]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def calls_path() -> str:
    """Where the compiled calls for this Python and torch lie."""
    import torch

    return os.path.join(HERE, f"_calls-py{sys.version_info[0]}.{sys.version_info[1]}-torch{torch.__version__}.so")


def build_calls(nvcc, force: bool = False) -> str:
    """Builds the compiled calls if they are stale.  They only save the host's time: where they do not compile (no C++
    compiler, no Python headers) this warns, leaves none behind, and the binding's Python form of them runs."""
    import torch

    target, src = calls_path(), os.path.join(CSRC, "calls.cpp")
    if torch.version.cuda is None:  # a torch without CUDA has nothing to call it with
        return target
    if not force and not _stale(target, [src, os.path.join(INCLUDE, "ringattn.h"), os.path.abspath(__file__)]):
        return target
    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"), sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")]
    tmp = target + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in include), src, "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = "" if r.returncode == 0 else f"{r.stdout}\n{r.stderr}" or f"status {r.returncode}"
    except OSError as e:
        failed = str(e)
    if failed:
        if os.path.exists(target):
            os.remove(target)
        warnings.warn(f"compiling calls.cpp failed, calls go through Python:\n{failed}", RuntimeWarning)
        return target
    os.replace(tmp, target)
    return target


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    deps = _deps()
    if not force and not _stale(LIB, deps):
        build_calls(nvcc)
        return LIB
    flags = NVCC_FLAGS + list(extra or [])

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        calls = ex.submit(build_calls, nvcc, force)
        objs = list(ex.map(compile_one, srcs))
        calls.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    extra = [a for a in sys.argv[1:] if a.startswith("-X") or a.startswith("--resource")]
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, extra=extra))

"""Build libw4a16.so from csrc/ with nvcc for sm_103a (in-tree, no cmake).

Each translation unit is compiled in parallel, then linked into one shared
library in ``_build/``.  Next to it goes a small extension module
(fastcall.cpp, host C++ against the installed torch's headers) that marshals
the arguments of the paged-cache calls; where it cannot be built, binding.py
does that itself, slower.  Host code is plain C++17 (portable between x86_64
and aarch64 hosts).  Floating point is IEEE: no fast-math, no flush-to-zero
(the CUDA-core kernel relies on subnormal FFMA operands).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libw4a16.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def flags() -> list:
    return [ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-Xcompiler", "-fvisibility=hidden", "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=true",
            "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) +
            [os.path.abspath(__file__)])


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in _deps())


FASTCALL_SRC = os.path.join(HERE, "fastcall.cpp")


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def _fastcall_flags():
    return ["-O1", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden"]


def fastcall_path():
    """The extension module's file (None without torch).  Its name holds what it
    has to agree with: torch, Python and machine, and the sources it is made of
    (their digest); so one made for something else, or before the C interface
    changed, is not found, and is never loaded."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return None
    with open(os.path.join(torch_dir, "version.py")) as f:
        found = re.search(r"^__version__ = ['\"]([^'\"]+)", f.read(), re.M)
    digest = hashlib.sha256(" ".join(_fastcall_flags()).encode())
    for source in (FASTCALL_SRC, os.path.join(INCLUDE, "w4a16.h")):
        with open(source, "rb") as f:
            digest.update(f.read())
    return os.path.join(BUILD_DIR, "_fastcall.%s.%s%s" % (found.group(1) if found else "unknown", digest.hexdigest()[:12],
                                                          sysconfig.get_config_var("EXT_SUFFIX")))


def build_fastcall(force: bool = False, verbose: bool = False):
    """The extension module's path, or None where it cannot be built."""
    path = fastcall_path()
    if path is None:
        return None
    if not force and os.path.exists(path):
        return path
    os.makedirs(BUILD_DIR, exist_ok=True)
    torch_dir, tmp = _torch_dir(), path + ".%d.tmp" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), *_fastcall_flags(),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"), "-I", INCLUDE, FASTCALL_SRC,
           "-o", tmp, "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        r = subprocess.CompletedProcess(cmd, 1, "", str(e))
    if r.returncode != 0:
        if verbose:
            print("fastcall.cpp not built:\n%s" % r.stderr)
        return None
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not is_stale():
        build_fastcall(verbose=verbose)
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc()] + flags() + list(extra_flags) + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        fastcall = ex.submit(build_fastcall, force, verbose)
        objs = list(ex.map(compile_one, srcs))
        fastcall.result()
    tmp = LIB_PATH + ".%d.tmp" % os.getpid()
    # static CUDA runtime (nvcc default): the library needs no libcudart at load time
    cmd = [nvcc(), ARCH, "-shared", "-Xcompiler", "-fPIC", "--cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

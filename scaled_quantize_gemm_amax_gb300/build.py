"""Build libfp8q.so in-tree: each .cu under csrc/ compiled by nvcc for sm_103a
(in parallel), then linked into one shared library next to this file; and beside it
_rowops.so, the Python extension of the row operators' allocation helpers (g++, the
installed torch's headers)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfp8q.so")
# The debug library: the same sources with FP8Q_DEBUG_INDEX, whose kernels check the
# index of their plain global accesses against the buffers' extents and report an
# access out of range through the device error word instead of making it.
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libfp8q_debug.so")
# The Python extension: host code only, the same for both libraries.
EXT_SOURCE = os.path.join(CSRC, "rowops_binding.cpp")
EXT = os.path.join(PKG, "_rowops.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-I", INCLUDE,
    "-Xptxas", "-warn-spills",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(INCLUDE, "fp8q.h"), os.path.abspath(__file__)]


def up_to_date(debug: bool = False) -> bool:
    lib = LIB_DEBUG if debug else LIB
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def start_extension(force: bool = False):
    """The compilation of _rowops.so under way: (process, temporary file, stamp), or None when it is up to date.

    The stamp, kept beside the object files, says what the extension was compiled against: it fits
    one version of torch and Python only."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    include = os.path.join(root, "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", INCLUDE, "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"), EXT_SOURCE,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    stamp = "\n".join((torch.__version__, sysconfig.get_config_var("EXT_SUFFIX") or "", *cmd))
    inputs = (EXT_SOURCE, os.path.join(INCLUDE, "fp8q.h"), os.path.abspath(__file__))
    if not force and os.path.exists(EXT) and all(os.path.getmtime(f) <= os.path.getmtime(EXT) for f in inputs) and \
            _read(_stamp_path()) == stamp:
        return None
    tmp = EXT + f".tmp{os.getpid()}"
    return subprocess.Popen([*cmd, "-o", tmp], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), tmp, stamp


def _stamp_path() -> str:
    return os.path.join(BUILD, os.path.basename(EXT) + ".stamp")


def _read(path: str) -> str | None:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _remove(path: str) -> None:
    if os.path.exists(path):
        os.remove(path)


def abandon_extension(started) -> None:
    """Wait for a compilation whose result is not wanted, and remove it."""
    if started is not None:
        started[0].terminate()
        started[0].communicate()
        _remove(started[1])


def finish_extension(started) -> None:
    if started is None:
        return
    p, tmp, stamp = started
    out, _ = p.communicate()
    if p.returncode != 0:
        sys.stderr.write(out)
        _remove(tmp)
        raise RuntimeError("g++ failed for rowops_binding.cpp")
    os.makedirs(BUILD, exist_ok=True)
    _remove(_stamp_path())   # never beside an extension that it does not describe
    os.replace(tmp, EXT)
    with open(_stamp_path(), "w") as f:
        f.write(stamp)


def _build_library(lib: str, verbose: bool, debug: bool) -> None:
    build_dir = BUILD_DEBUG if debug else BUILD
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(build_dir, os.path.basename(src).replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, *NVCC_FLAGS, *(["-DFP8Q_DEBUG_INDEX"] if debug else []), "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stderr.write(out)
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(os.path.basename(f) for f in failed))
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.run([nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", *objs, "-o", tmp], check=True)
    os.replace(tmp, lib)


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    lib = LIB_DEBUG if debug else LIB
    extension = start_extension(force)
    if not force and up_to_date(debug):
        finish_extension(extension)
        return lib
    try:
        _build_library(lib, verbose, debug)
    except BaseException:
        abandon_extension(extension)
        raise
    finish_extension(extension)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))

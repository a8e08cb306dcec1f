"""Build liborpo_head.so in-tree with nvcc for sm_103a (GB300).

Each .cu file is compiled in parallel into an object, then linked into a shared
library against the shared CUDA runtime (the one PyTorch also loads).  The
result lives in ``orpo_preference_loss_gb300/_build/`` (git-ignored).  The Python
module of csrc/binding.cpp is compiled beside it with the host compiler, against
PyTorch's headers; where that fails there is a warning, and the calls it is for go through
ctypes.  Either is skipped when it is newer than its sources and headers.

``build(debug=True)`` makes the bounds-checked variant ``liborpo_head_debug.so``
in ``_build_debug/``: the same sources with ORPO_DEBUG_BOUNDS, where every
computed index is checked against its buffer and a miss is reported in the
status word (ORPO_STATUS_BOUNDS) instead of touching memory.
"""

from __future__ import annotations

import fcntl
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB_NAME = "liborpo_head.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
DEBUG_OUT_DIR = os.path.join(PKG, "_build_debug")
DEBUG_LIB_PATH = os.path.join(DEBUG_OUT_DIR, "liborpo_head_debug.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-O2", "-Xptxas", "-v"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build liborpo_head")


def binding_path(debug: bool = False) -> str:
    """The Python module, named for the PyTorch and Python that it is compiled against: it fits no other."""
    import torch

    return os.path.join(DEBUG_OUT_DIR if debug else OUT_DIR, f"orpo_binding-{torch.__version__}-{sys.implementation.cache_tag}.so")


def _binding_command(out: str):
    """The host compiler's command for the Python module (its library is handed to it when it is loaded)."""
    import torch

    home = os.path.dirname(torch.__file__)
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"), "-I", os.path.join(home, "include"), "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", os.path.join(CSRC, "binding.cpp"), "-o", out,
            "-L", os.path.join(home, "lib"), f"-Wl,-rpath,{os.path.join(home, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(path: str, sources) -> bool:
    """Whether path is there and no older than its sources, the C ABI's headers and this file."""
    deps = [*sources, *glob.glob(os.path.join(ROOT, "include", "*.h")), os.path.abspath(__file__)]
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def _library_up_to_date(debug: bool) -> bool:
    return _newer(DEBUG_LIB_PATH if debug else LIB_PATH,
                  [*_sources(), *glob.glob(os.path.join(CSRC, "*.cuh")), *glob.glob(os.path.join(CSRC, "*.h"))])


def _binding_up_to_date(debug: bool) -> bool:
    return _newer(binding_path(debug), [os.path.join(CSRC, "binding.cpp")])


def up_to_date(debug: bool = False) -> bool:
    return _library_up_to_date(debug) and _binding_up_to_date(debug)


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile the library if needed; returns the path of the shared object.

    Safe to call from several processes at once (ranks of one job): a file lock lets one of them
    build while the others wait and then find the library up to date."""
    lib, out = (DEBUG_LIB_PATH, DEBUG_OUT_DIR) if debug else (LIB_PATH, OUT_DIR)
    if not force and up_to_date(debug):
        return lib
    os.makedirs(out, exist_ok=True)
    with open(os.path.join(out, ".build.lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        try:
            if not force and up_to_date(debug):
                return lib
            with ThreadPoolExecutor(max_workers=1) as ex:
                binding = None if not force and _binding_up_to_date(debug) else ex.submit(_build_binding, verbose, debug)
                if force or not _library_up_to_date(debug):
                    _build_locked(verbose, debug)
                failed = binding is not None and binding.result()
            if failed:
                sys.stderr.write(f"--- the compiler failed on binding.cpp\n{failed}\n")
                warnings.warn(f"{os.path.basename(binding_path(debug))} could not be built: the calls that it is for go through ctypes, "
                              "which takes some microseconds more each", RuntimeWarning, stacklevel=2)
            return lib
        finally:
            fcntl.flock(lock, fcntl.LOCK_UN)


def _build_binding(verbose: bool, debug: bool) -> str | None:
    """Returns what the compiler said where it failed."""
    path = binding_path(debug)
    tmp = path + ".tmp"
    try:
        r = subprocess.run(_binding_command(tmp), capture_output=True, text=True)
        failed, said = r.returncode != 0, f"{r.stdout}\n{r.stderr}"
    except OSError as e:  # no compiler
        failed, said = True, str(e)
    if failed:
        for old in (path, tmp):  # one of an earlier build may not fit the library any more
            if os.path.exists(old):
                os.remove(old)
        return said
    if verbose:
        sys.stderr.write(f"--- binding.cpp\n{said}\n")
    os.replace(tmp, path)
    return None


def _build_locked(verbose: bool, debug: bool) -> str:
    nvcc = nvcc_path()
    srcs = _sources()
    lib, out = (DEBUG_LIB_PATH, DEBUG_OUT_DIR) if debug else (LIB_PATH, OUT_DIR)
    flags = NVCC_FLAGS + (["-DORPO_DEBUG_BOUNDS"] if debug else [])
    objs = [os.path.join(out, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = [nvcc, *ARCH, *flags, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r

    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        results = list(ex.map(compile_one, zip(srcs, objs)))
    failed = False
    for src, r in results:
        if r.returncode != 0:
            failed = True
            sys.stderr.write(f"--- nvcc failed on {src}\n{r.stdout}\n{r.stderr}\n")
        elif verbose:
            sys.stderr.write(f"--- {os.path.basename(src)}\n{r.stderr}")
    if failed:
        raise RuntimeError("liborpo_head build failed")
    tmp = lib + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"liborpo_head link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))

"""Build libswa.so in-tree: nvcc for sm_103a, translation units compiled in parallel.

`build(checked=True)` builds libswa_checked.so from the same sources with
SWA_CHECKS=1: its kernels test every global load and store against the
extent of its tensor and report an access outside it as SWA_ERR_BOUNDS
instead of making it (include/swa.h, swa_workspace_status).  It is a
testing build; nothing loads it unless asked to (swa.checked_lib())."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libswa.so")
CHECKED_BUILD_DIR = os.path.join(PKG, "_build_checked")
CHECKED_LIB_PATH = os.path.join(PKG, "libswa_checked.so")
# the CPython extension that calls the rotary and paged-cache entry points on torch tensors
BIND_SOURCE = "swa_bind.cpp"
SOURCES = ["swa_api.cpp", "swa_fwd.cu", "swa_fwd_pair.cu", "swa_bwd_dkv.cu", "swa_bwd_dq.cu", "swa_aux.cu",
           "swa_noalloc.cu", "swa_host.cpp", "swa_rope.cu", "swa_paged_rows.cu", "swa_paged_tile.cu", "swa_paged.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libswa")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "swa.h")]
    return [f for f in files if os.path.isfile(f)]


def is_stale(lib_path: str = LIB_PATH) -> bool:
    if not os.path.exists(lib_path):
        return True
    t = os.path.getmtime(lib_path)
    return any(os.path.getmtime(f) > t for f in _inputs())


def bind_path() -> str:
    """Where the CPython extension of the installed torch and the running Python
    is: it is linked against the C++ ABI of both, so after an upgrade of either it
    counts as not built."""
    try:
        import torch

        version = torch.__version__
    except ImportError:
        version = "none"
    return os.path.join(PKG, f"_swa_bind.torch-{version}{sysconfig.get_config_var('EXT_SUFFIX') or '.so'}")


def build_bind(verbose: bool = False) -> str:
    """Compile the CPython extension against the installed torch; returns its path."""
    import torch

    path = bind_path()

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           os.path.join(CSRC, BIND_SOURCE), "-o", tmp, "-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BIND_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def _bind_failure(verbose: bool):
    """Build the extension; the exception where that fails, None where it does not."""
    try:
        build_bind(verbose)
    except Exception as e:
        return e
    return None


def _report(failure) -> None:
    if failure is None:
        return
    path = bind_path()
    if is_stale(path) and os.path.exists(path):
        os.remove(path)  # its structs may not be the library's
    warnings.warn(f"the Python calls of the rotary and paged operators are not available: {failure}", RuntimeWarning,
                  stacklevel=3)


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Compile every translation unit for sm_103a and link libswa.so (or,
    with `checked`, the bounds-checked libswa_checked.so); returns its path.

    The library needs nvcc alone.  The CPython extension is built beside it and
    needs PyTorch's C++ headers: where that fails the library is complete, a
    RuntimeWarning says why, and the calls that go through the extension raise
    ImportError."""
    lib_path = CHECKED_LIB_PATH if checked else LIB_PATH
    build_dir = CHECKED_BUILD_DIR if checked else BUILD_DIR
    bind = force or is_stale(bind_path())
    if not force and not is_stale(lib_path):
        if bind:
            _report(_bind_failure(verbose))
        return lib_path
    nvcc = _nvcc()
    os.makedirs(build_dir, exist_ok=True)
    defines = ["-DSWA_CHECKS=1"] if checked else []

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *defines, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        pending = ex.submit(_bind_failure, verbose) if bind else None
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib_path + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    if pending is not None:
        _report(pending.result())
    return lib_path


if __name__ == "__main__":
    print(build(force=True, verbose=True))

"""Build libbq.so (the C-ABI CUDA library) in-tree for sm_100a, and the
extension module _torch_calls.so that calls it on torch tensors.

Each csrc/*.cu file is compiled by nvcc (in parallel) into _build/, then
linked into block_scaled_w8a8_b200/libbq.so with the CUDA runtime linked
statically, so the library loads on hosts without a GPU.  csrc/torch_calls.cpp
is compiled by the host compiler against torch's headers and linked to libbq.so.

    python -m block_scaled_w8a8_b200.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbq.so")
EXT = os.path.join(PKG, "_torch_calls.so")
EXT_STAMP = os.path.join(BUILD, "_torch_calls.stamp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
# No fast-math, no flush-to-zero: quantisation must round like IEEE fp32.
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libbq")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime():
    ts = [os.path.getmtime(os.path.join(CSRC, f)) for f in os.listdir(CSRC)]
    ts.append(os.path.getmtime(os.path.join(ROOT, "include", "bq.h")))
    ts.append(os.path.getmtime(__file__))
    return max(ts)


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _compile_ext() -> str:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "torch_calls.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(cuda, "include"), "-I" + os.path.join(ROOT, "include"),
           "-c", os.path.join(CSRC, "torch_calls.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling torch_calls.cpp failed:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_ext(obj: str):
    import torch
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libbq.so",
           "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking _torch_calls failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def _ext_stamp() -> str:
    """What the extension fits besides its sources: the interpreter and torch."""
    try:
        import torch
    except ImportError:
        return ""
    return f"python {sysconfig.get_config_var('SOABI')}, torch {torch.__version__}\n"


def _fresh(path: str) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()


def _ext_fresh() -> bool:
    if not _fresh(EXT) or not os.path.exists(EXT_STAMP):
        return False
    with open(EXT_STAMP) as f:
        return f.read() == _ext_stamp()


def _build_ext():
    try:
        _link_ext(_compile_ext())
        with open(EXT_STAMP, "w") as f:
            f.write(_ext_stamp())
    except (ImportError, OSError, RuntimeError) as e:
        # the C ABI and the calls through ctypes do not need it; those that do raise.  An
        # old one would call the new library with the old arguments.
        for f in (EXT, EXT_STAMP):
            if os.path.exists(f):
                os.remove(f)
        warnings.warn(f"{os.path.basename(EXT)} is not built (norm, rotary positions, cache and "
                      f"attention cannot be called on torch tensors): {e}", RuntimeWarning,
                      stacklevel=3)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Build what is out of date; raises if libbq.so cannot be built, warns if the
    extension module (host compiler, torch's headers) cannot."""
    lib, ext = force or not _fresh(LIB), force or not _ext_fresh()
    if not lib and not ext:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    if lib:
        srcs = sources()
        with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
            objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if ext:
        _build_ext()
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose_ptxas=args.verbose_ptxas))

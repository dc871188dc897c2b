"""Builds the sm_103a shared library in-tree with nvcc.

The library is a plain C-ABI ``.so`` (see ``include/gqa_decode.h``,
``include/gqa_shared_keys.h`` and ``include/gqa_paged.h``); nothing in it links
against PyTorch.  Beside it stands the native binding of the paged calls
(``csrc/paged_binding.cpp``, g++), which does, and only marshals tensors.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
HEADER = os.path.join(ROOT, "include", "gqa_decode.h")
SHARED_KEYS_HEADER = os.path.join(ROOT, "include", "gqa_shared_keys.h")
PAGED_HEADER = os.path.join(ROOT, "include", "gqa_paged.h")
LIB = os.path.join(PKG, "libgqa_decode_sm103.so")
# The same library with device-side bounds checks (-DGQA_DEBUG): every
# global write of the decode kernel, the rows kernel and its merges, and the
# kernels around a paged cache is checked against its buffer and skipped if
# outside it, every TMA tile origin against its tensor, reads of a page table
# and of a tree's bits against their rows; each shows as GQA_ERR_BOUNDS from gqa_decode_get_error.  For testing only.
DEBUG_LIB = os.path.join(PKG, "libgqa_decode_sm103_debug.so")
# The same library with the decode kernel's clock64 event trace
# (-DGQA_TRACE): gqa_trace_attach() names a device buffer that the following
# launches stamp per CTA, role and block.  For measurement only.
TRACE_LIB = os.path.join(PKG, "libgqa_decode_sm103_trace.so")
BINDING_SOURCE = os.path.join(CSRC, "paged_binding.cpp")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh", ".h"))] + [
        HEADER, SHARED_KEYS_HEADER, PAGED_HEADER]


def binding_path() -> str:
    """Where the binding for the present Python and PyTorch is: it holds for no others."""
    import torch

    return os.path.join(PKG, f"_paged_binding-{sys.implementation.cache_tag}-torch{torch.__version__}.so")


def _binding_includes():
    """Include directories of the binding, or None where PyTorch, or its headers or
    Python's, are not installed."""
    try:
        import torch
    except (ImportError, OSError):
        return None
    base = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)), "include")
    python = sysconfig.get_paths()["include"]
    for header in (os.path.join(python, "Python.h"), os.path.join(base, "torch", "csrc", "autograd", "python_variable.h")):
        if not os.path.exists(header):
            return None
    return [python, base, os.path.join(base, "torch", "csrc", "api", "include"),
            os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")]


def _start_binding(out: str, includes) -> subprocess.Popen:
    import torch

    base = os.path.dirname(os.path.abspath(torch.__file__))
    return subprocess.Popen([
        shutil.which("g++") or "g++", "-O2", "-std=c++20", "-shared", "-fPIC", "-w",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *(f"-I{i}" for i in includes),
        BINDING_SOURCE, "-L" + os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
        "-o", out])


def _binding_up_to_date(out: str) -> bool:
    if not os.path.exists(out):
        return False
    return all(os.path.getmtime(s) <= os.path.getmtime(out) for s in (BINDING_SOURCE, HEADER, PAGED_HEADER))


def up_to_date(out: str = LIB) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(s) <= t for s in sources())


# Translation units: the host sides (C ABI, planning, merge kernels) of the three
# headers, one unit per head_dim and merge mode holding that combination's
# decode kernels and one per head_dim and place of the keys with its rows
# kernels, compiled in parallel and linked into one shared library.
INSTANCES = [(hd, cl) for hd in (64, 128, 256) for cl in (0, 1)]


def _units(build_dir: str):
    units = [(os.path.join(CSRC, f"{name}.cu"), [], os.path.join(build_dir, f"{name}.o"))
             for name in ("gqa_decode", "gqa_shared_keys", "gqa_paged")]
    for hd in (64, 128, 256):
        for paged in (0, 1):
            units.append((os.path.join(CSRC, "rows_instances.cu"),
                          [f"-DGQA_INST_HD={hd}", f"-DGQA_INST_PAGED={paged}"],
                          os.path.join(build_dir, f"rows_{hd}_{paged}.o")))
    for hd, cl in INSTANCES:
        units.append((os.path.join(CSRC, "decode_instances.cu"), [f"-DGQA_INST_HD={hd}", f"-DGQA_INST_CLUSTER={cl}"],
                      os.path.join(build_dir, f"decode_{hd}_{cl}.o")))
    return units


def build(force: bool = False, out: str = LIB, extra_flags=(), verbose: bool = False) -> str:
    """Compile the csrc translation units for sm_103a (in parallel) and link
    them into ``out``, and for the library itself the binding beside it (each
    skipped if current).  Without PyTorch or its headers or Python's the C library
    is built alone, with a warning: the Python functions of
    ``include/gqa_paged.h`` then raise."""
    if out != LIB:
        return _build_library(force, out, extra_flags, verbose)
    includes = _binding_includes()
    if includes is None:
        warnings.warn("PyTorch, its headers or Python's are not installed: the binding of the paged calls is not built")
        return _build_library(force, out, extra_flags, verbose)
    binding = binding_path()
    if not force and _binding_up_to_date(binding):
        return _build_library(force, out, extra_flags, verbose)
    os.makedirs(os.path.join(PKG, "_build"), exist_ok=True)
    temporary = os.path.join(PKG, "_build", f"{os.path.basename(binding)}.{os.getpid()}")
    process = _start_binding(temporary, includes)
    try:
        _build_library(force, out, extra_flags, verbose)
    finally:
        failed = process.wait() != 0  # waited for in either case
    if failed:
        raise subprocess.CalledProcessError(process.returncode, "g++ (paged_binding.cpp)")
    os.replace(temporary, binding)
    return out


def _build_library(force: bool, out: str, extra_flags, verbose: bool) -> str:
    if not force and up_to_date(out):
        return out
    build_dir = os.path.join(os.path.dirname(os.path.abspath(out)), "_build",
                             os.path.splitext(os.path.basename(out))[0])
    os.makedirs(build_dir, exist_ok=True)
    base = [_nvcc(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-I", os.path.join(ROOT, "include"), *extra_flags]
    if verbose:
        base.insert(1, "-Xptxas=-v")
    procs = []
    for src, defs, obj in _units(build_dir):
        procs.append((obj, subprocess.Popen([*base, *defs, "-c", src, "-o", obj])))
    failed = [obj for obj, p in procs if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, f"nvcc ({', '.join(os.path.basename(f) for f in failed)})")
    subprocess.run([_nvcc(), ARCH, "-shared", *[obj for obj, _ in procs], "-o", out + ".tmp"], check=True)
    os.replace(out + ".tmp", out)
    return out


def build_debug(force: bool = False) -> str:
    """The -DGQA_DEBUG build of the library (bounds-checked), beside the other."""
    return build(force=force, out=DEBUG_LIB, extra_flags=("-DGQA_DEBUG",))


def build_trace(force: bool = False) -> str:
    """The -DGQA_TRACE build of the library (event stamps), beside the other."""
    return build(force=force, out=TRACE_LIB, extra_flags=("-DGQA_TRACE",))


if __name__ == "__main__":
    print(build(force=True, verbose=True))

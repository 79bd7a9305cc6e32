"""Builds the CUDA library ``libfa_attention.so`` in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel, then linked into one shared
object next to this file.  A rebuild happens when a source or header is newer
than the library.  Usage: ``python -m exact_attention_37_gb300.build [-v] [-f] [--debug]``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfa_attention.so")
OBJDIR = os.path.join(HERE, "_build")
# The native marshalling module of the Python binding (host code only).
BINDING = os.path.join(HERE, "_native.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
# The debug build: the same sources with -DFA_DEBUG (device-side bounds, alignment
# and barrier-phase checks that record into the device error record, never trap).
LIB_DEBUG = os.path.join(HERE, "libfa_attention_debug.so")
OBJDIR_DEBUG = os.path.join(HERE, "_build_debug")
SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_bwd_sq.cu", "fa_bwd256.cu", "fa_selftest.cu", "fa_host.cu",
           "fa_rule.cu", "fa_kv4.cu", "fa_kv4_attend.cu"]
# Compiled once for each kind of score rule (FA_RULE_KIND: with or without a bias, a cap, ids).
RULE_SOURCES = ["fa_fwd_rule.cu", "fa_bwd_sq_rule.cu", "fa_bwd256_rule.cu"]
RULE_KINDS = range(8)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the attention library")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "fa_attention.h"))
    return files


def _flags_file(objdir: str) -> str:
    return os.path.join(objdir, "flags.txt")


def up_to_date(lib: str = LIB, objdir: str = OBJDIR, flags=()) -> bool:
    """The library exists, is newer than every source, and was built with `flags`."""
    if not os.path.exists(lib):
        return False
    try:
        with open(_flags_file(objdir)) as f:
            if f.read() != " ".join(flags):
                return False
    except OSError:
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build_binding(force: bool = False) -> str:
    """Compile the binding's native module against the installed torch if needed; returns its path."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    flags_file = os.path.join(OBJDIR, "binding.txt")
    inputs = [BINDING_SOURCE, os.path.join(INCLUDE, "fa_attention.h")]
    key = f"{torch.__version__} {sysconfig.get_python_version()}"
    if not force and os.path.exists(BINDING) and os.path.exists(flags_file):
        with open(flags_file) as f:
            if f.read() == key and all(os.path.getmtime(x) <= os.path.getmtime(BINDING) for x in inputs):
                return BINDING
    os.makedirs(OBJDIR, exist_ok=True)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
           "-I", sysconfig.get_paths()["include"], BINDING_SOURCE, "-o", tmp, "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the native binding did not compile:\n" + r.stderr)
    os.replace(tmp, BINDING)
    with open(flags_file, "w") as f:
        f.write(key)
    return BINDING


def build(verbose: bool = False, force: bool = False, extra_flags=(), debug: bool = False,
          nvtx: bool | None = None) -> str:
    """Compile and link the library (and the binding's native module) if needed; returns its path.  ``debug`` builds
    the checked variant (``libfa_attention_debug.so``) instead; ``nvtx`` (default:
    the FA_NVTX environment variable is set to 1) marks every C-ABI call with an
    NVTX range."""
    lib, objdir = (LIB_DEBUG, OBJDIR_DEBUG) if debug else (LIB, OBJDIR)
    if nvtx is None:
        nvtx = os.environ.get("FA_NVTX") == "1"
    extra_flags = (*extra_flags, *(["-DFA_DEBUG"] if debug else []), *(["-DFA_NVTX"] if nvtx else []))
    if not force and up_to_date(lib, objdir, extra_flags):
        build_binding()
        return lib
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()

    def compile_one(unit):
        src, kind = unit
        obj = os.path.join(objdir, src.replace(".cu", ".o" if kind is None else f"_{kind}.o"))
        kind_flags = [] if kind is None else [f"-DFA_RULE_KIND={kind}"]
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, *kind_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    units = [(s, k) for s in RULE_SOURCES for k in RULE_KINDS] + [(s, None) for s in SOURCES]
    with cf.ThreadPoolExecutor(max_workers=max(4, os.cpu_count() or 4)) as ex:
        binding = ex.submit(build_binding, force)
        results = list(ex.map(compile_one, units))
        binding.result()
    errors = []
    for src, obj, r in results:
        if verbose and (r.stdout or r.stderr):
            print(f"--- {src}\n{r.stdout}{r.stderr}", file=sys.stderr)
        if r.returncode != 0:
            errors.append(f"{src}:\n{r.stderr}")
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    tmp = lib + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[obj for _, obj, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, lib)
    with open(_flags_file(objdir), "w") as f:
        f.write(" ".join(extra_flags))
    return lib


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv, debug="--debug" in sys.argv))

"""Builds libar.so (the C-ABI library) in-tree with nvcc for sm_103a.

The translation units compile in parallel, then link into one shared
library next to this file.  Nothing is installed anywhere else.

A second library, libar_test.so, is the same code with the test hooks
compiled in (AR_TEST_HOOKS: the launch-shape override, the fault injection
of the bounded-wait tests and the programmatic-launch switch, each read from
the environment, and a communicator over local buffers for the peer
barrier's timeout test).  Only ar_api.cu, ar_peer.cu and ar_cache_api.cu
differ, so only they are compiled twice.
_binding-*.so is the CPython extension that marshals the paged key-value cache
calls from torch tensors (host code only, compiled by g++ against torch's
headers; its name tells torch's and Python's versions).  Where it cannot be built the other calls, which do not need it, are
built all the same.

The tests of forced launch shapes and of bounded waits, and the shape sweeps
that build the AUTO table, load it; everything else loads libar.so, which
reads no environment variable.
"""
from __future__ import annotations

import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libar.so")
TEST_LIB = os.path.join(PKG, "libar_test.so")
BINDING_SOURCE = os.path.join(CSRC, "ar_binding.cpp")

SOURCES = ["ar_api.cu", "ar_kern_f32.cu", "ar_kern_f16.cu", "ar_kern_bf16.cu", "ar_noalloc.cu", "ar_host.cu",
           "ar_peer.cu", "ar_cache_api.cu", "ar_append.cu", "ar_pages.cu", "ar_attn_f32.cu", "ar_attn_f16.cu", "ar_attn_bf16.cu",
           "ar_tree_f32.cu", "ar_tree_f16.cu", "ar_tree_bf16.cu"]
HEADERS = ["ar_internal.h", "ar_kernels.cuh", "ar_tma.cuh", "ar_lamport.cuh", "ar_launch.cuh", "ar_launch_k.cuh",
           "ar_auto_table.h", "ar_cache.h", "ar_layers.h", "ar_split.h", "ar_attn.cuh", "ar_tree.h", "ar_tree.cuh",
           "ar_tcgen05.cuh", "ar_tree_mma.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libar.so")
    return exe


def binding_path() -> str:
    """The extension module of this Python and torch, whose C++ interfaces it is compiled against: one of other versions has
    another name, and is neither loaded nor taken for built."""
    return os.path.join(PKG, f"_binding-torch{torch.__version__}{importlib.machinery.EXTENSION_SUFFIXES[0]}")


def _older(outputs: list, deps: list) -> bool:
    """Whether an output is missing or older than what it is made of."""
    if not all(os.path.exists(f) for f in outputs):
        return True
    t = min(os.path.getmtime(f) for f in outputs)
    return any(os.path.getmtime(d) > t for d in [*deps, os.path.join(INCLUDE, "ar.h"), __file__])


def _stale() -> bool:
    return _older([LIB, TEST_LIB], [os.path.join(CSRC, f) for f in SOURCES + HEADERS])


def _binding_stale() -> bool:
    return _older([binding_path()], [BINDING_SOURCE])


def _binding_command(out: str) -> list:
    """The g++ command of the extension module: torch's own headers and libraries, and CUDA's for its stream type."""
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_path("include")]
    lib_dir = os.path.join(root, "lib")
    return [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in includes), BINDING_SOURCE,
            "-o", out, f"-L{lib_dir}", f"-Wl,-rpath,{lib_dir}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10_cuda", "-lc10"]


def _start(cmd: list, verbose: bool) -> subprocess.Popen:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _succeeded(p: subprocess.Popen, show: bool) -> bool:
    """Waits for a compiler; its output is shown where asked for, or where it failed."""
    out, _ = p.communicate()
    if out and (show or p.returncode != 0):
        print(out, file=sys.stderr)
    return p.returncode == 0


def _build_library(verbose: bool, ptxas_info: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    units = [(src, os.path.join(BUILD, src.replace(".cu", ".o")), []) for src in SOURCES]
    hooked = ["ar_api.cu", "ar_peer.cu", "ar_cache_api.cu"]
    units += [(src, os.path.join(BUILD, src.replace(".cu", "_test.o")), ["-DAR_TEST_HOOKS"]) for src in hooked]
    for src, obj, defs in units:
        cmd = [cc, *ARCH, *FLAGS, *defs, "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, _start(cmd, verbose)))
        objs.append(obj)
    failed = [src for src, p in procs if not _succeeded(p, verbose or ptxas_info)]
    if failed:
        raise RuntimeError(f"nvcc failed on {failed}")
    product = objs[:len(SOURCES)]
    swap = {os.path.join(BUILD, src.replace(".cu", ".o")): obj for src, obj in zip(hooked, objs[len(SOURCES):])}
    test = [swap.get(o, o) for o in product]
    for lib, lib_objs in ((LIB, product), (TEST_LIB, test)):
        tmp = f"{lib}.{os.getpid()}.tmp"
        subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *lib_objs], check=True)
        os.replace(tmp, lib)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libar.so, libar_test.so and the extension module where a source is newer; returns libar.so's path.

    An extension module that cannot be built is warned of, and an older one taken away: the calls that go through it then
    raise, all others work.
    """
    made, binding, tmp = True, None, f"{binding_path()}.{os.getpid()}.tmp"
    if force or _binding_stale():
        try:
            binding = _start(_binding_command(tmp), verbose)   # beside the library's units
        except Exception as e:   # no compiler, or none of torch's headers
            print(e, file=sys.stderr)
            made = False
    try:
        if force or _stale():
            _build_library(verbose, ptxas_info)
    finally:
        if binding is not None:
            made = _succeeded(binding, verbose)
            if made:
                os.replace(tmp, binding_path())
    if not made:
        if os.path.exists(binding_path()):
            os.remove(binding_path())
        warnings.warn("the extension module could not be compiled: ar_kv_append, ar_kv_compact, ar_kv_copy_pages, "
                      "ar_paged_attention, ar_tree_attention and ar_attention_join are not available from Python")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB)

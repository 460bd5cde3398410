"""Builds libar.so (the C-ABI library) in-tree with nvcc for sm_103a.

The translation units compile in parallel, then link into one shared
library next to this file.  Nothing is installed anywhere else.

A second library, libar_test.so, is the same code with the test hooks
compiled in (AR_TEST_HOOKS: the launch-shape override, the fault injection
of the bounded-wait tests and the programmatic-launch switch, each read from
the environment, and a communicator over local buffers for the peer
barrier's timeout test).  Only ar_api.cu and ar_peer.cu differ, so only
they are compiled twice.
_binding.so is the CPython extension that marshals the paged key-value cache
calls from torch tensors (host code only, compiled by g++ against torch's
headers).

The tests of forced launch shapes and of bounded waits, and the shape sweeps
that build the AUTO table, load it; everything else loads libar.so, which
reads no environment variable.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libar.so")
TEST_LIB = os.path.join(PKG, "libar_test.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "ar_binding.cpp")

SOURCES = ["ar_api.cu", "ar_kern_f32.cu", "ar_kern_f16.cu", "ar_kern_bf16.cu", "ar_noalloc.cu", "ar_host.cu",
           "ar_peer.cu", "ar_cache_api.cu", "ar_append.cu", "ar_attn_f32.cu", "ar_attn_f16.cu", "ar_attn_bf16.cu"]
HEADERS = ["ar_internal.h", "ar_kernels.cuh", "ar_tma.cuh", "ar_lamport.cuh", "ar_launch.cuh", "ar_launch_k.cuh",
           "ar_auto_table.h", "ar_cache.h", "ar_attn.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libar.so")
    return exe


def _stale() -> bool:
    if not all(os.path.exists(f) for f in (LIB, TEST_LIB, BINDING)):
        return True
    t = min(os.path.getmtime(f) for f in (LIB, TEST_LIB, BINDING))
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "ar.h"), BINDING_SOURCE, __file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_command(out: str) -> list:
    """The g++ command of the extension module: torch's own headers and libraries, and CUDA's for its stream type."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_path("include")]
    lib_dir = os.path.join(root, "lib")
    return [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in includes), BINDING_SOURCE,
            "-o", out, f"-L{lib_dir}", f"-Wl,-rpath,{lib_dir}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10_cuda", "-lc10"]


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libar.so, libar_test.so and _binding.so if any source is newer; returns libar.so's path."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    units = [(src, os.path.join(BUILD, src.replace(".cu", ".o")), []) for src in SOURCES]
    units.append(("ar_api.cu", os.path.join(BUILD, "ar_api_test.o"), ["-DAR_TEST_HOOKS"]))
    units.append(("ar_peer.cu", os.path.join(BUILD, "ar_peer_test.o"), ["-DAR_TEST_HOOKS"]))
    for src, obj, defs in units:
        cmd = [cc, *ARCH, *FLAGS, *defs, "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        objs.append(obj)
    binding = f"{BINDING}.{os.getpid()}.tmp"
    cmd = _binding_command(binding)
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    procs.append(("ar_binding.cpp", subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or ptxas_info or p.returncode != 0):
            print(out, file=sys.stderr)
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"the compiler failed on {failed}")
    os.replace(binding, BINDING)
    product = objs[:len(SOURCES)]
    swap = {os.path.join(BUILD, "ar_api.o"): objs[-2], os.path.join(BUILD, "ar_peer.o"): objs[-1]}
    test = [swap.get(o, o) for o in product]
    for lib, lib_objs in ((LIB, product), (TEST_LIB, test)):
        tmp = f"{lib}.{os.getpid()}.tmp"
        subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *lib_objs], check=True)
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB)

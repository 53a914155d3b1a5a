"""Build the CUDA library libar_gb300.so in-tree, for sm_103a only.

Each translation unit is compiled by nvcc in parallel into ``_build/`` and
linked into ``libar_gb300.so`` next to this file; the Python binding of the
feed-forward operators is compiled beside them by the host compiler, against
torch's headers, into ``_ops.so``, which loads that library.  Usage:
``python -m shot_allreduce_ranks_gb300.build [--force]``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libar_gb300.so")
OPS = os.path.join(PKG, "_ops.so")

SOURCES = ["ar_api.cu", "k_oneshot.cu", "k_oneshot_bulk.cu", "k_twophase.cu", "k_fused_ll8.cu",
           "k_rs_ag.cu", "op_api.cu", "k_gemm_any.cu", "k_gemm_tc.cu",
           "k_gemm_mid.cu", "k_gemm_i8.cu", "k_gemm_few.cu", "k_rows.cu", "k_dropout.cu"]
HEADERS = [os.path.join(CSRC, "ar_internal.cuh"), os.path.join(CSRC, "ops_internal.cuh"),
           os.path.join(CSRC, "tc_device.cuh"),
           os.path.join(INCLUDE, "ar.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# No fast math: IEEE fp32 adds with subnormals kept, no contraction.
NVCC_FLAGS = ARCH + [
    "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=false",
    "-I", INCLUDE, "-I", CSRC,
]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return path


def ops_commands(obj: str, out: str):
    """Compile and link commands of the operators' Python binding."""
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    libs = os.path.join(home, "lib")
    return [
        [cxx, "-std=c++20", "-O2", "-fPIC", "-fvisibility=hidden", "-Wno-deprecated-declarations",
         "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
         "-I", INCLUDE, "-isystem", os.path.join(home, "include"), "-isystem", sysconfig.get_paths()["include"],
         "-isystem", os.path.join(cuda, "include"), "-c", os.path.join(CSRC, "py_ops.cpp"), "-o", obj],
        [cxx, "-shared", "-o", out, obj, "-L", PKG, "-l:" + os.path.basename(LIB), "-L", libs, "-lc10", "-lc10_cuda",
         "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs],
    ]


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + HEADERS):
            jobs.append([nvcc(), *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o])
    ops_src, ops_obj = os.path.join(CSRC, "py_ops.cpp"), os.path.join(BUILD, "py_ops.o")
    ops_tmp = OPS + ".tmp%d" % os.getpid()
    compile_ops, link_ops = ops_commands(ops_obj, ops_tmp)
    if force or _stale(ops_obj, [ops_src, os.path.join(INCLUDE, "ar.h")]):
        jobs.insert(0, compile_ops)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n%s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if force or _stale(OPS, [ops_obj]):
        run(link_ops)
        os.replace(ops_tmp, OPS)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

"""Build libestream.so in-tree with nvcc for sm_103a.

Compiles each CUDA translation unit in parallel (one -gencode, no fast-math)
and links them with the shared CUDA runtime into
``routed_expert_ffn_topk_gb300/libestream.so``, and the compiled part of the
binding (plain C, Python's own headers) into ``_binding.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libestream.so")
BINDING_PATH = os.path.join(PKG, "_binding.so")
SOURCES = ["route.cu", "route_static.cu", "expert_gemm.cu", "expert_f32.cu", "runtime.cu",
           "pipeline_model.cu", "router.cu", "decode.cu", "mx4.cu", "mx4_product.cu", "kv_append.cu",
           "kv_attend.cu", "sample.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(OBJ_DIR, exist_ok=True)
    headers = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh")))
    headers.append(os.path.join(INCLUDE, "estream.h"))
    common = [nvcc, *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "-I" + INCLUDE, "-I" + CSRC]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJ_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append(common + ["-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("the compiler failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)

    binding = os.path.join(CSRC, "binding.c")
    python_include = sysconfig.get_paths()["include"]
    # without Python's headers the binding takes its interpreted way alone
    if os.path.exists(os.path.join(python_include, "Python.h")) and (
            force or _stale(BINDING_PATH, [binding, os.path.join(INCLUDE, "estream.h")])):
        tmp_binding = BINDING_PATH + ".tmp%d" % os.getpid()
        run([shutil.which("gcc") or "cc", "-O2", "-std=c11", "-Wall", "-Wextra", "-fPIC", "-shared", "-I" + INCLUDE,
             "-I" + python_include, binding, "-o", tmp_binding])
        os.replace(tmp_binding, BINDING_PATH)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            list(ex.map(run, jobs))
    if force or jobs or _stale(LIB_PATH, objs):
        libdir = _cuda_lib_dir(nvcc)
        tmp = LIB_PATH + ".tmp%d" % os.getpid()
        run([nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
             "-Xlinker", "-rpath=" + libdir, "-L" + libdir])
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))

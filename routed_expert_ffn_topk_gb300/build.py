"""Build libestream.so in-tree with nvcc for sm_103a.

Compiles each CUDA translation unit in parallel (one -gencode, no fast-math)
and links them with the shared CUDA runtime into
``routed_expert_ffn_topk_gb300/libestream.so``, and the compiled part of the
binding (plain C, Python's own headers) into ``_binding`` with this interpreter's
suffix.
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
BINDING_PATH = os.path.join(PKG, "_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
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


def _compile(cmd, verbose: bool = False) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the compiler failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)


def build_binding(path: str = BINDING_PATH, python_include: str | None = None, force: bool = False,
                  verbose: bool = False) -> None:
    """The compiled part of the binding; without Python's headers there is none, and the binding takes its
    interpreted way alone. What an import would find in its stead (a file without this interpreter's tag, or of an
    older source) is removed."""
    python_include = sysconfig.get_paths()["include"] if python_include is None else python_include
    source = os.path.join(CSRC, "binding.c")
    untagged = os.path.join(os.path.dirname(path), "_binding.so")
    if untagged != path and os.path.exists(untagged):
        os.remove(untagged)
    if not force and not _stale(path, [source, os.path.join(INCLUDE, "estream.h")]):
        return
    if not os.path.exists(os.path.join(python_include, "Python.h")):
        if os.path.exists(path):
            os.remove(path)
        return
    tmp = path + ".tmp%d" % os.getpid()
    _compile([shutil.which("gcc") or "cc", "-O2", "-std=c11", "-Wall", "-Wextra", "-fPIC", "-shared", "-I" + INCLUDE,
              "-I" + python_include, source, "-o", tmp], verbose)
    os.replace(tmp, path)


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

    build_binding(force=force, verbose=verbose)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            list(ex.map(lambda cmd: _compile(cmd, verbose), jobs))
    if force or jobs or _stale(LIB_PATH, objs):
        libdir = _cuda_lib_dir(nvcc)
        tmp = LIB_PATH + ".tmp%d" % os.getpid()
        _compile([nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
                  "-Xlinker", "-rpath=" + libdir, "-L" + libdir], verbose)
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))

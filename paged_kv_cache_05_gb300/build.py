"""Build libpagedkv.so in-tree with nvcc for sm_103a (no cmake, no setuptools).

Each translation unit compiles in parallel; the objects are linked into
``paged_kv_cache_05_gb300/libpagedkv.so`` against the shared CUDA runtime.
``_pkvbind.so`` beside it is the Python module of the grouped entry points
(g++ against the installed torch's headers).
Usage: ``python -m paged_kv_cache_05_gb300.build [--force] [--verbose]``.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
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
LIB = os.path.join(PKG, "libpagedkv.so")
BIND = os.path.join(PKG, "_pkvbind.so")
BIND_SOURCE = "binding.cpp"
SOURCES = ["errors.cu", "cache_ops.cu", "decode_api.cu", "decode_f16.cu", "decode_bf16.cu",
           "decode_shared_f16.cu", "decode_shared_bf16.cu", "decode_append_f16.cu",
           "decode_append_bf16.cu", "decode_noalloc.cu", "decode_grouped.cu", "prefill.cu",
           "prefill_grouped_f16.cu", "prefill_grouped_bf16.cu", "prefill_cut_f16.cu",
           "prefill_cut_bf16.cu", "prefill_grouped_api.cu",
           "rope_cache.cu", "block_manager.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _flags(src: str, verbose: bool):
    common = ["-O3", "-std=c++17", "-I", INCLUDE, "-I", CSRC, "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall"]
    if src.endswith(".cu"):
        extra = ARCH + ["-lineinfo", "--expt-relaxed-constexpr"]
        if verbose:
            extra += ["-Xptxas", "-v"]
        return common + extra
    return common


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "pagedkv.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def up_to_date() -> bool:
    deps = _deps_mtime()
    return all(os.path.exists(f) and os.path.getmtime(f) >= deps for f in (LIB, BIND))


def _cuda_home(cc: str) -> str:
    return os.environ.get("CUDA_HOME") or os.path.dirname(os.path.dirname(os.path.realpath(cc)))


def _bind_commands(cc: str, out: str):
    """Compile and link commands of the binding module."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found (the binding is compiled against its headers)")
    torch = os.path.dirname(spec.origin)
    cxx = os.environ.get("CXX") or "g++"
    obj = os.path.join(BUILD, "binding.o")
    inc = [INCLUDE, os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(_cuda_home(cc), "include"), sysconfig.get_paths()["include"]]
    comp = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall"]
    for i in inc:
        comp += ["-isystem" if "torch" in i else "-I", i]
    comp += ["-c", os.path.join(CSRC, BIND_SOURCE), "-o", obj]
    tl = os.path.join(torch, "lib")
    link = [cxx, "-shared", obj, "-o", out, "-L", tl, "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", "-L", PKG, "-l:libpagedkv.so", "-Wl,-rpath,$ORIGIN:" + tl]
    return comp, link


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc] + _flags(src, verbose) + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compile failed: %s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
        return obj, r.stdout + r.stderr

    def run(cmd, what):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("%s failed: %s\n%s%s" % (what, " ".join(cmd), r.stdout, r.stderr))

    tmp_bind = BIND + ".tmp.%d" % os.getpid()
    bind_compile, bind_link = _bind_commands(cc, tmp_bind)
    with cf.ThreadPoolExecutor(max_workers=jobs or len(SOURCES) + 1) as ex:
        bound = ex.submit(run, bind_compile, "compile")
        results = list(ex.map(compile_one, SOURCES))
        bound.result()
    if verbose:
        for _, log in results:
            if log.strip():
                sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = ([cc, "-shared", "-cudart", "shared"] + ARCH + objs
           + ["-Xlinker", "-rpath=$ORIGIN:/usr/local/cuda/lib64", "-o", tmp])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed: %s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
    os.replace(tmp, LIB)
    run(bind_link, "link")
    os.replace(tmp_bind, BIND)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))

"""Build libpa.so (the C-ABI CUDA library) in-tree for sm_103a.

Each source under csrc/ (.cu kernels and the host-only block manager .cpp)
is compiled by nvcc in parallel, then linked into
paged_kv_cache_284_gb300/libpa.so.  Objects go to _build/ (git-ignored).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpa.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
SOURCES = ["pa_api.cu", "pa_write_kv.cu", "pa_plan.cu", "pa_plan_window.cu", "pa_short.cu",
           "pa_long.cu", "pa_long_window.cu", "pa_window.cu", "pa_merge.cu", "pa_static.cu",
           "pa_rope.cu", "pa_copy.cu", "pa_build.cu", "pa_linear.cu",
           "pa_linear_prompt.cu", "pa_blocks.cpp", "pa_shard.cpp"]
BINDING = "pa_torch.cpp"  # -> _pa_torch.so, host code that reads torch's tensors
BINDING_LIB = os.path.join(PKG, "_pa_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "--expt-relaxed-constexpr", "-I", INCLUDE] + list(extra)


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_job(out: str):
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_path("include"), os.path.join(os.path.dirname(os.path.dirname(_nvcc())),
                                                       "include"), INCLUDE]
    lib = os.path.join(root, "lib")
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", os.path.join(CSRC, BINDING),
             "-o", out] + [x for d in inc for x in ("-I", d)] +
            ["-L", lib, "-Wl,-rpath," + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
             "-ltorch_python"], os.path.join(root, "version.py"))


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libpa.so, and the binding of its small calls; returns
    libpa.so's path."""
    nvcc = _nvcc()
    os.makedirs(OBJ, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    headers += [os.path.join(INCLUDE, h) for h in os.listdir(INCLUDE) if h.endswith(".h")]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, "-c", s, "-o", o] + _flags(extra_flags))
    tmp_binding = BINDING_LIB + f".tmp{os.getpid()}"
    binding, torch_version = _binding_job(tmp_binding)
    headers_c = [h for h in headers if h.endswith(".h")]
    bind = force or _stale(BINDING_LIB, [os.path.join(CSRC, BINDING), torch_version] + headers_c)
    cuda_jobs = bool(jobs)
    if bind:
        jobs.append(binding)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        errors = [(c, r) for c, r in zip(jobs, results) if r.returncode != 0]
        for c, r in zip(jobs, results):
            if verbose or r.returncode != 0:
                print(" ".join(c[:6]), "\n", r.stdout, r.stderr)
        if errors:
            raise RuntimeError(f"compiling failed: {[' '.join(c[:6]) for c, _ in errors]}")
    if bind:
        os.replace(tmp_binding, BINDING_LIB)
    if force or cuda_jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, "-shared", "-o", tmp] + objs + ARCH + [
            "-cudart", "shared", "-Xlinker", "-rpath,/usr/local/cuda/lib64"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            print(r.stdout, r.stderr)
            raise RuntimeError("link of libpa.so failed")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

"""Builds libkvp.so in-tree for sm_103a with nvcc (no cmake, no torch
extension machinery) and _calls.so, the binding's argument checks in C++, with
g++ against the installed torch's headers.  Translation units compile in
parallel, then link.  The library needs neither torch nor Python's headers:
where _calls.so cannot be built, a warning says why, and the calls that need it
raise.

    python -m paged_prefix_shared_decode_gb300.build [--force]
"""
from __future__ import annotations

import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkvp.so")
CALLS = os.path.join(HERE, "_calls.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]

SOURCES = ["pool.cpp", "radix.cpp", "plan.cpp", "attn_kernels.cu", "attn_tc.cu", "kv_kernels.cu", "kv4_kernels.cu", "no_alloc.cu",
           "mass_kernels.cu", "mass_tc.cu", "evict_kernels.cu", "draft_verify.cu", "rope_kernels.cu", "page_kernels.cu",
           "sparse_attn.cu", "beam_kernels.cu"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _flags(src: str) -> list:
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if src.endswith(".cu"):
        return common + ARCH + ["-lineinfo", "--expt-relaxed-constexpr"]
    return common


def _stale(target: str, deps: list) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _calls_job(force: bool, headers: list):
    """The command that compiles _calls.so and where it writes to, or None if
    the module is up to date (with the sources and with the torch installed).
    Raises ModuleNotFoundError without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise ModuleNotFoundError("No module named 'torch'")
    torch = list(spec.submodule_search_locations)[0]
    version = runpy.run_path(os.path.join(torch, "version.py"))["__version__"]
    src = os.path.join(CSRC, "py_calls.cpp")
    stamp = os.path.join(OUT_DIR, "calls_torch_version")
    built = open(stamp).read() if os.path.exists(stamp) else ""
    if not force and built == version and not _stale(CALLS, [src] + headers):
        return None
    tmp = CALLS + f".{os.getpid()}.tmp"
    lib = os.path.join(torch, "lib")
    cmd = [os.environ.get("CXX") or "g++", "-shared", "-O2", "-std=c++17", "-fPIC", src, "-o", tmp,
           f'-DKVP_TORCH_VERSION="{version}"', "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(torch, "include"), "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    return cmd, tmp, stamp, version


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(INCLUDE, "kvp.h"))
    objs = []
    jobs = []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(OUT_DIR, s + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc, "-c", src, "-o", obj] + _flags(s)
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    def build_calls():
        job = _calls_job(force, headers)
        if job is None:
            return ""
        cmd, tmp, stamp, version = job
        try:
            err = run(cmd)
        except (OSError, RuntimeError):
            if os.path.exists(CALLS):
                os.remove(CALLS)      # (of other sources or another torch)
            raise
        os.replace(tmp, CALLS)
        with open(stamp, "w") as f:
            f.write(version)
        return err

    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        calls = ex.submit(build_calls)
        for err in ex.map(run, jobs):
            if verbose and err:
                print(err)
    try:
        err = calls.result()
        if verbose and err:
            print(err)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"_calls.so is not built: {e}")
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        run([nvcc, "-shared", "-o", tmp] + objs + ARCH + ["-lcudart"])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))

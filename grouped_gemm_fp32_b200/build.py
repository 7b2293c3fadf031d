"""Build ``libmoe.so`` (the C-ABI CUDA library) in-tree with nvcc for sm_100a, and
``libmoe_debug.so``, the same sources with MOE_DEBUG=1 (device-side checks of the
group table and tile coordinates that report MOE_ERR_BAD_ROUTING instead of
following a bad entry; loaded instead of libmoe.so when MOE_LIB_DEBUG=1), and with g++
``_bind.so``, the Python calls of the operators around the layer (csrc/bind.cpp).

    python -m grouped_gemm_fp32_b200.build [--force]
"""
from __future__ import annotations

import glob
import importlib.metadata
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe.so")
BIND = os.path.join(HERE, "_bind.so")
BIND_ABI = os.path.join(HERE, "_bind.abi")  # the Python and torch that _bind.so is built for
LIB_DEBUG = os.path.join(HERE, "libmoe_debug.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        [os.path.join(INCLUDE, "moe.h"), os.path.abspath(__file__)]


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in deps())


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _build_one(lib: str, extra, force: bool, verbose: bool):
    """The sources side by side (a few at a time), then one link."""
    if not force and not stale(lib):
        return
    tmp = lib + f".tmp{os.getpid()}"
    flags = [f for f in NVCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.basename(s)[:-3] + ".o") for s in sources()]

        def one(src, obj):
            cmd = [nvcc(), *flags, *extra, "-I", INCLUDE, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.check_call(cmd)

        # the largest first: they take longest
        jobs = sorted(zip(sources(), objs), key=lambda j: -os.path.getsize(j[0]))
        with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as pool:
            for r in [pool.submit(one, *j) for j in jobs]:
                r.result()
        subprocess.check_call([nvcc(), *NVCC_FLAGS, "-o", tmp, *objs])
    os.replace(tmp, lib)


def _bind_abi() -> str:
    """What _bind.so is built against besides its sources."""
    return f"{sys.implementation.cache_tag} torch {importlib.metadata.version('torch')}"


def bind_stale() -> bool:
    newest = max(map(os.path.getmtime, (os.path.join(CSRC, "bind.cpp"),
                                        os.path.join(INCLUDE, "moe.h"), os.path.abspath(__file__))))
    if not os.path.exists(BIND) or os.path.getmtime(BIND) < newest:
        return True
    try:
        with open(BIND_ABI) as f:
            return f.read() != _bind_abi()
    except OSError:
        return True


def _build_bind(force: bool, verbose: bool):
    if not force and not bind_stale():
        return
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           os.path.join(CSRC, "bind.cpp"), "-o", tmp, "-L", os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, BIND)
    with open(BIND_ABI, "w") as f:
        f.write(_bind_abi())


def build(force: bool = False, verbose: bool = False, debug: bool = True) -> str:
    """Both libraries (the debug one unless ``debug`` is False) and the binding; returns
    libmoe.so's path."""
    jobs = [(_build_one, LIB, [], force, verbose), (_build_bind, force, verbose)]
    if debug:
        jobs.append((_build_one, LIB_DEBUG, ["-DMOE_DEBUG=1"], force, verbose))
    with ThreadPoolExecutor(len(jobs)) as pool:
        for r in [pool.submit(*j) for j in jobs]:
            r.result()
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)

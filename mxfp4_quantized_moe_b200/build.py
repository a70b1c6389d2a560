"""Builds the in-tree shared libraries with nvcc (sm_100a only).

* ``libmxfp4_moe.so``: the library.
* ``libmxfp4_moe_debug.so``: the same sources with ``-DMXFP4_MOE_DEBUG=1``: kernels check the
  indices they read from the workspace and record MXFP4_MOE_ERR_DEVICE_BOUNDS instead of
  making the access (``mxfp4_moe_build_flags`` reports the build).  Loaded instead of the
  library when ``MXFP4_MOE_LIBRARY=debug``.
* ``_edge.<torch>.<python>.so``: the host side of the operators at the block's edge as a CPython
  module (csrc/binding.cpp), which calls whichever of the two is loaded.  It is compiled against
  the headers of one torch and one Python, and its name says which: under others it is built anew,
  not loaded.

Usage: ``python -m mxfp4_quantized_moe_b200.build [--verbose-ptxas]`` builds all three.  Cross-compiles
without a GPU.  The libraries statically link the CUDA runtime, so they load on a machine
without a driver (calls then fail with MXFP4_MOE_ERR_CUDA).
"""

from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmxfp4_moe.so")
LIB_DEBUG = os.path.join(HERE, "libmxfp4_moe_debug.so")
BINDING_SOURCE = os.path.join("csrc", "binding.cpp")
BINDING = os.path.join(HERE, f"_edge.torch-{importlib.metadata.version('torch')}."
                             f"{sysconfig.get_config_var('SOABI')}.so")
SOURCES = ["csrc/api.cu", "csrc/grouped_gemm.cu", "csrc/kernels_small.cu",
           "csrc/forward_static.cu", "csrc/selftest.cu", "csrc/residual_router.cu",
           "csrc/routing.cu", "csrc/norm.cu"]
DEPS = SOURCES + ["csrc/common.cuh", "csrc/kernels.h", "csrc/aux_kernels.h", "csrc/block_edge.h"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(HERE, d) for d in DEPS] + [os.path.join(ROOT, "include", "mxfp4_moe.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, ptxas_verbose: bool = False, debug: bool = False) -> str:
    """The library (or its debug build) and, beside it, the binding module."""
    with ThreadPoolExecutor(max_workers=2) as pool:
        beside = pool.submit(build_binding, force and not debug)
        lib = build_library(force, ptxas_verbose, debug)
        beside.result()
    return lib


def build_library(force: bool = False, ptxas_verbose: bool = False, debug: bool = False) -> str:
    lib = LIB_DEBUG if debug else LIB
    if not force and not needs_build(lib):
        return lib
    flags = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a",
             "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
             "-I", os.path.join(ROOT, "include")]
    if debug:
        flags += ["-DMXFP4_MOE_DEBUG=1"]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]

    def run(cmd):
        r = subprocess.run([nvcc(), *cmd], cwd=HERE, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    # one compiler per source, then the link (no device code crosses a file)
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
            said = list(pool.map(lambda so: run([*flags, "-c", "-o", so[1],
                                                 os.path.join(HERE, so[0])]), zip(SOURCES, objects)))
        run(["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", lib + ".tmp", *objects])
    if ptxas_verbose:
        sys.stderr.write("".join(said))
    os.replace(lib + ".tmp", lib)
    return lib


def needs_binding() -> bool:
    deps = (os.path.join(HERE, BINDING_SOURCE), os.path.join(ROOT, "include", "mxfp4_moe.h"))
    return not os.path.exists(BINDING) or any(os.path.getmtime(d) > os.path.getmtime(BINDING)
                                              for d in deps)


def build_binding(force: bool = False) -> str:
    """The host-side module `_edge` (C++ against torch's headers; no device code)."""
    if not force and not needs_binding():
        return BINDING
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-shared", "-fPIC",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in (os.path.join(at, "include"),
                                os.path.join(at, "include", "torch", "csrc", "api", "include"),
                                os.path.join(cuda, "include"), sysconfig.get_paths()["include"])),
           "-o", BINDING + ".tmp", os.path.join(HERE, BINDING_SOURCE), "-L" + os.path.join(at, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, cwd=HERE, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the binding failed to compile:\n" + r.stdout + r.stderr)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build_all(force: bool = False, ptxas_verbose: bool = False) -> list[str]:
    with ThreadPoolExecutor(max_workers=3) as pool:
        every = [pool.submit(build_library, force, ptxas_verbose),
                 pool.submit(build_library, force, False, True),
                 pool.submit(build_binding, force)]
        return [b.result() for b in every]


if __name__ == "__main__":
    print("\n".join(build_all(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv)))

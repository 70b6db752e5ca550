"""Ahead-of-time build of the gfx950 GEMM library (``libmi355_gemm.so``) and of
the Python extension that calls the block operators in it (``_block.so``).

Each HIP translation unit is compiled by ``hipcc --offload-arch=gfx950`` into
an object (in parallel), then linked into one shared library next to this
file. Packed fp32 VALU ops are disabled for all device code.
"""
from __future__ import annotations

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
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libmi355_gemm.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
BIND_PATH = os.path.join(PKG, "_block.so")
BIND_SOURCE = "block_bind.cpp"

SOURCES = ["gemm_api.cpp", "kernels_generic.hip", "kernels_wholek.hip", "kernels_f32.hip",
           "kernels_f16.hip", "kernels_bf16.hip", "kernels_f8.hip", "kernels_mxf8.hip",
           "kernels_mxf4.hip", "block_api.cpp", "kernels_mx4.hip", "kernels_moe.hip",
           "kernels_norm.hip"]

ARCH = "gfx950"


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build the GEMM library)")


def common_flags():
    return ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", "-Wall",
            "-Wno-unused-function", "-Xclang", "-target-feature", "-Xclang",
            "-packed-fp32-ops", "-I", INCLUDE, "-I", CSRC]


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj] + \
        common_flags() + list(extra)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {src} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _bind() -> None:
    """The extension: host code against torch's headers, linked to the library."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    lib = os.path.join(torch, "lib")
    tmp = BIND_PATH + ".tmp"
    cmd = [hipcc(), "-x", "c++", os.path.join(CSRC, BIND_SOURCE), "-x", "none", LIB_PATH, "-o", tmp, "-O2",
           "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",   # which torch's headers ask for
           "-I", INCLUDE, "-I", os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include"),
           "-I", os.path.join(torch, "include"),
           "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-L", lib, "-lc10", "-lc10_hip", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building {BIND_SOURCE} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND_PATH)


def build(jobs: int = 0, extra=(), verbose: bool = False, only=None) -> str:
    """Compile every HIP source for gfx950 and link the shared library.
    ``only`` (a list of source names) recompiles just those and links the
    others' existing objects."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    todo = list(SOURCES) if only is None else [s for s in SOURCES if s in only]
    objs = {s: os.path.join(BUILD_DIR, os.path.splitext(s)[0] + ".o") for s in SOURCES
            if s not in todo}
    for s, o in objs.items():
        if not os.path.exists(o):
            raise RuntimeError(f"no object for {s}: build it first")
    jobs = jobs or min(len(SOURCES), max(1, (os.cpu_count() or 4)))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        futs = {ex.submit(_compile, s, extra): s for s in todo}
        for f in cf.as_completed(futs):
            objs[futs[f]] = f.result()
            if verbose:
                print(f"compiled {futs[f]}", flush=True)
    tmp = LIB_PATH + ".tmp"
    cmd = [hipcc(), "-shared", f"--offload-arch={ARCH}", "-fPIC", f"-Wl,-soname,{LIB_NAME}", "-o", tmp] + \
        [objs[s] for s in SOURCES]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if only is None or BIND_SOURCE in only:
        _bind()
    return LIB_PATH


if __name__ == "__main__":
    args = sys.argv[1:]
    only = [a for a in args if a in SOURCES + [BIND_SOURCE]] or None
    print(build(verbose=True, extra=[a for a in args if a not in SOURCES + [BIND_SOURCE]], only=only))

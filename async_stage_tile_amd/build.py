"""Build the tile-stream library for gfx950 with hipcc, in-tree.

libpipetile.so -- all kernels + the C ABI of include/pipe_tile.h (the tile stream)
and include/pipe_linear.h (the quantised linear layer's operators).

_linear.so -- the linear layer's Python marshalling in C++ (csrc/linear_binding.cpp,
host code against the installed torch's headers; the Python wrappers work
without it, slower). Where it cannot be built (no torch, no headers, no C++
compiler) the build says so and goes on without it.

Every translation unit compiles to its own object, in parallel; the stream
kernel source is compiled once per group of stage counts. Then the library
is linked and moved into place atomically.

Usage: python -m async_stage_tile_amd.build  (or build() from Python).
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
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpipetile.so")
BINDING = os.path.join(PKG, "_linear.so")
ARCH = "gfx950"

# (source, object, extra defines)
UNITS = [
    ("pipe_api.hip", "pipe_api.o", []),
    ("pipe_stream_aux.hip", "pipe_stream_aux.o", []),
    ("pipe_stream.hip", "pipe_stream_s1_2.o", ["PIPE_STREAM_STAGES_LO=1", "PIPE_STREAM_STAGES_HI=2"]),
    ("pipe_stream.hip", "pipe_stream_s3_4.o", ["PIPE_STREAM_STAGES_LO=3", "PIPE_STREAM_STAGES_HI=4"]),
    ("pipe_stream.hip", "pipe_stream_s5_6.o", ["PIPE_STREAM_STAGES_LO=5", "PIPE_STREAM_STAGES_HI=6"]),
    ("pipe_stream.hip", "pipe_stream_s7_8.o", ["PIPE_STREAM_STAGES_LO=7", "PIPE_STREAM_STAGES_HI=8"]),
    ("pipe_unified.hip", "pipe_unified.o", []),
    ("pipe_gemm.hip", "pipe_gemm_ring.o", ["PIPE_GEMM_PART=1"]),
    ("pipe_gemm.hip", "pipe_gemm_unified.o", ["PIPE_GEMM_PART=2"]),
    ("pipe_linear_api.hip", "pipe_linear_api.o", []),
    ("pipe_norm.hip", "pipe_norm.o", []),
    ("pipe_gemm_fp8.hip", "pipe_gemm_fp8.o", []),
    ("pipe_gemm_w4.hip", "pipe_gemm_w4.o", []),
    ("pipe_layernorm.hip", "pipe_layernorm.o", []),
    ("pipe_mx_quant.hip", "pipe_mx_quant.o", []),
    ("pipe_gemm_mx.hip", "pipe_gemm_mx.o", []),
]
# Kept for callers that list the tile-stream sources.
SOURCES = sorted({u[0] for u in UNITS})


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain is required to build libpipetile.so")


def compile_command(src: str, obj: str, defines: list) -> list:
    return [
        hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-c",
        # Packed fp32 VALU forms are kept out of the generated code.
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-I", os.path.join(ROOT, "include"),
        *[f"-D{d}" for d in defines],
        os.path.join(CSRC, src), "-o", obj,
    ]


def link_command(objs: list, out: str) -> list:
    return [hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", *objs, "-o", out]


def _run(cmd: list, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        what = next((a for a in cmd if a.endswith((".hip", ".cpp"))), cmd[-1])
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed with exit code {res.returncode}: {what}")


def _link(units: list, out: str, verbose: bool) -> None:
    objs = [os.path.join(OBJ, o) for (_, o, _) in units]
    tmp = out + ".tmp"
    _run(link_command(objs, tmp), verbose)
    os.replace(tmp, out)


def build_binding(verbose: bool = False) -> None:
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no C++ compiler found: one is required to build _linear.so")
    tmp = BINDING + ".tmp"
    _run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", sysconfig.get_paths()["include"], "-I", os.path.join(t, "include"),
          "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
          "-L", os.path.join(t, "lib"), "-o", tmp, os.path.join(CSRC, "linear_binding.cpp"),
          "-ltorch_python", "-ltorch_cpu", "-lc10"], verbose)
    os.replace(tmp, BINDING)


def build(verbose: bool = False, jobs: int | None = None) -> str:
    os.makedirs(OBJ, exist_ok=True)
    units = UNITS
    jobs = jobs or min(len(units) + 1, max(1, min(8, os.cpu_count() or 1)))
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        futs = [ex.submit(_run, compile_command(s, os.path.join(OBJ, o), d), verbose)
                for (s, o, d) in units]
        binding = ex.submit(build_binding, verbose)
        for f in futs:
            f.result()
    _link(UNITS, LIB, verbose)
    if binding.exception() is not None:
        # One of an earlier build may not fit this library.
        if os.path.exists(BINDING):
            os.remove(BINDING)
        sys.stderr.write(f"warning: _linear.so was not built ({binding.exception()}); "
                         "the linear layer's calls take the Python wrappers\n")
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))

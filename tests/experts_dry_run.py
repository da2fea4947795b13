"""The grouped and 4-bit products' host code without a GPU: grouped_*.hip and
w4_*.hip compiled for the host alone and linked with mx_dry_run's stand-in for
the runtime, which records each launch and runs nothing.  Pointers are never
dereferenced."""
import concurrent.futures as cf
import ctypes
import os
import re
import subprocess

from dense_gemm_row_amd import build, grouped, w4
from tests.mx_dry_run import STAND_IN, DryRun

# The dense product that many rows of activations take after dequantisation.
DENSE = r"""
#define DENSE(name, value) extern "C" gemm_status_t name(int64_t, int64_t, int64_t, const uint16_t*, int64_t, const uint16_t*, \
    int64_t, uint16_t*, int64_t, void* stream, const gemm_config_t*) { \
  launches.push_back(Launch{#name, {1, 1}, 1, stream, {0, 0, 0, 0}}); return GEMM_OK; }
DENSE(gemm_bf16_bt, 0)
DENSE(gemm_f16_bt, 0)
"""
KERNELS = ("gemm_bf16_bt", "gemm_f16_bt", "matmul_pipe", "wgrad_pipe", "matmul_general", "wgrad_general", "matmul_few",
           "dequantize_rows", "quantize_rows", "quantize_cols")


def kernel(launch):
    """The launched kernel's own name."""
    return next(k for k in KERNELS if k in launch.name.decode())


def tile(launch):
    """The side of a pipelined kernel's tile and its LDS stages."""
    return tuple(map(int, re.search(r"4TileILb\dELb\dELi(\d+)ELi\d+ELi\d+ELi\d+ELi(\d)", launch.name.decode()).groups()))


def compile_dry(folder: str) -> DryRun:
    objs = [o for o in build.OBJECTS if o[0].startswith(("grouped_", "w4_"))]

    def one(o):
        src, stem, defines = o
        out = os.path.join(folder, stem + ".o")
        subprocess.run([build.hipcc(), f"--offload-arch={build.ARCH}", "--offload-host-only", "-O1", "-std=c++17", "-fPIC",
                        "-fwrapv", "-Wno-unused-function", "-I", build.INCLUDE, "-I", build.CSRC, *defines, "-c",
                        os.path.join(build.CSRC, src), "-o", out], check=True, capture_output=True)
        return out

    with cf.ThreadPoolExecutor(min(len(objs), os.cpu_count() or 1)) as ex:
        outs = list(ex.map(one, objs))
    undefined = subprocess.run(["nm", "-u", *outs], check=True, capture_output=True, text=True).stdout
    images = sorted(set(re.findall(r"__hip_fatbin\w*", undefined)))
    shim = os.path.join(folder, "stand_in.cc")
    with open(shim, "w") as f:
        f.write(STAND_IN + DENSE + "".join(f'extern "C" {{ char {s}[16]; }}\n' for s in images))
    out = os.path.join(folder, "libdry.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,--no-undefined", "-I", build.INCLUDE, shim, *outs,
                    "-o", out], check=True, capture_output=True)
    L = ctypes.CDLL(out)
    for module in (grouped, w4):
        for name in module.EXPORTS:  # (the signatures of the bindings)
            ours, theirs = getattr(L, name), getattr(module.lib(), name)
            ours.argtypes, ours.restype = theirs.argtypes, theirs.restype
    return DryRun(L)

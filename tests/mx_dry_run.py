"""The microscaled operators' host code without a GPU: mx_*.hip compiled for
the host alone and linked with a stand-in for the runtime that records each
launch and runs nothing, so that tests can look at grids at sizes that no
memory holds (sums that leave their type wrap around, so that they show).
Nothing of HIP's runtime is loaded; pointers are never
dereferenced."""
import concurrent.futures as cf
import ctypes
import os
import re
import subprocess

from dense_gemm_row_amd import build, gemm

STAND_IN = r"""
#include <stdint.h>
#include <string.h>
#include <map>
#include <string>
#include <vector>
#include "gemm.h"
struct Dim { unsigned x, y, z; };
struct Launch { const char* name; unsigned grid[2], block; void* stream; int64_t arg[4]; };
static std::map<const void*, std::string>& names() { static std::map<const void*, std::string> m; return m; }
static std::vector<Launch> launches;
static Dim g_grid, g_block;
static size_t g_lds;
static void* g_stream;
namespace gemm {
gemm_status_t set_last_error(gemm_status_t st, const char*) { return st; }
}
extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* h; return &h; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, Dim*, Dim*, int*) {
  names()[host] = name;
}
int __hipPushCallConfiguration(Dim g, Dim b, size_t lds, void* s) { g_grid = g; g_block = b; g_lds = lds; g_stream = s; return 0; }
int __hipPopCallConfiguration(Dim* g, Dim* b, size_t* lds, void** s) { *g = g_grid; *b = g_block; *lds = g_lds; *s = g_stream; return 0; }
int hipLaunchKernel(const void* f, Dim g, Dim b, void** args, size_t, void* stream) {
  Launch l = {names()[f].c_str(), {g.x, g.y}, b.x, stream, {0, 0, 0, 0}};
  // The integers behind the structure of arguments.
  const struct { const char* kernel; const char* sizes; } known[] = {
      {"matmul_direct", "48"}, {"wgrad_general", "48"}, {"quantize_rows", "444"}, {"quantize_cols", "44"}};
  for (auto& k : known)
    if (strstr(l.name, k.kernel))
      for (int i = 0; k.sizes[i]; ++i)
        l.arg[i] = k.sizes[i] == '8' ? *(const int64_t*)args[i + 1] : *(const int*)args[i + 1];
  launches.push_back(l);
  return 0;
}
// (An error ends a call that launches without end.)
int hipGetLastError() { return launches.size() < 4096 ? 0 : 1; }
const char* hipGetErrorString(int) { return ""; }
void dry_clear() { launches.clear(); }
int dry_count() { return (int)launches.size(); }
const Launch* dry_get(int i) { return &launches[i]; }
}
"""


class Launch(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("grid", ctypes.c_uint * 2), ("block", ctypes.c_uint), ("stream", ctypes.c_void_p),
                ("arg", ctypes.c_int64 * 4)]

    @property
    def kernel(self):
        """The kernel's own name."""
        return next(k for k in ("matmul_direct", "matmul_skinny", "matmul_pipe", "wgrad_general", "wgrad_pipe", "split_planes",
                                "reduce_partials", "dequantize_rows", "dequantize_cols", "quantize_rows", "quantize_cols")
                    if k in self.name.decode())


class DryRun:
    def __init__(self, lib):
        self.lib = lib
        lib.dry_get.restype = ctypes.POINTER(Launch)

    def __call__(self, name, *args):
        """(status, launches) of one call of the C-ABI."""
        self.lib.dry_clear()
        status = getattr(self.lib, name)(*args)
        return status, [Launch.from_buffer_copy(self.lib.dry_get(i).contents) for i in range(self.lib.dry_count())]


def compile_dry(folder: str) -> DryRun:
    objs = [o for o in build.OBJECTS if o[0].startswith("mx_")]

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
        f.write(STAND_IN + "".join(f'extern "C" {{ char {s}[16]; }}\n' for s in images))
    out = os.path.join(folder, "libdry.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,--no-undefined", "-I", build.INCLUDE, shim, *outs,
                    "-o", out], check=True, capture_output=True)
    L = ctypes.CDLL(out)
    i64, i32, p, f = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
    L.gemm_mx_quantize.argtypes = L.gemm_mx_dequantize.argtypes = [i32, i32, i32, i64, i64] + [p, i64] * 3 + [p]
    L.gemm_mx_matmul.argtypes = [i32, i64, i64, i64] + [p, i64] * 5 + [p, ctypes.POINTER(gemm.GemmEpilogue)]
    L.gemm_mx_matmul_values.argtypes = [i32, i32, i64, i64, i64] + [p, i64] * 5 + [p, ctypes.POINTER(gemm.GemmEpilogue)]
    L.gemm_mx_wgrad.argtypes = [i32, i32, i64, i64, i64] + [p, i64] * 4 + [f, f, p, i64, p]
    L.gemm_mx_wgrad_workspace_bytes.argtypes = [i32, i64, i64, i64]
    L.gemm_mx_wgrad_workspace_bytes.restype = i64
    return DryRun(L)

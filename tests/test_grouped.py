"""Grouped products on the host: exports, refusals before any launch, the
arithmetic of segments and tiles.  CPU only."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest

from dense_gemm_row_amd import build, gemm, grouped

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PO, PX, PW, PY = 0x08000000, 0x10000000, 0x40000000, 0x80000000  # never dereferenced
OK, INVALID, UNSUPPORTED, ALIAS = (gemm.GEMM_OK, gemm.GEMM_ERR_INVALID_ARG, gemm.GEMM_ERR_UNSUPPORTED,
                                   gemm.GEMM_ERR_ALIAS)
F32, F16, BF16, F8 = gemm.DTYPE_F32, gemm.DTYPE_F16, gemm.DTYPE_BF16, gemm.DTYPE_F8


def test_exports_its_header():
    text = open(os.path.join(ROOT, "include", "gemm_grouped.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(grouped.EXPORTS)
    for n in names:
        assert hasattr(grouped.lib(), n) and hasattr(grouped, n)


def product(dtype=BF16, c=BF16, trans=0, G=4, T=64, N=48, K=32, offsets=PO, X=PX, ldx=32, W=PW, ldw=48, stride=48 * 32,
            Y=PY, ldy=48, fill=1):
    return grouped.gemm_grouped_matmul(dtype, c, trans, G, T, N, K, offsets, X, ldx, W, ldw, stride, Y, ldy, fill)


def wgrad(dtype=BF16, c=F32, G=4, T=64, K=32, N=48, offsets=PO, X=PX, ldx=32, dY=PY, ldy=48, dW=PW, ldw=48, stride=48 * 32,
          alpha=1.0, beta=0.0):
    return grouped.gemm_grouped_wgrad(dtype, c, G, T, K, N, offsets, X, ldx, dY, ldy, dW, ldw, stride, alpha, beta)


@pytest.mark.parametrize("fn", [product, wgrad])
@pytest.mark.parametrize("kw, want", [
    (dict(dtype=F8), INVALID), (dict(dtype=-1), INVALID), (dict(c=F16), INVALID), (dict(c=7), INVALID),
    (dict(dtype=F32, c=BF16), INVALID),
    (dict(G=-1), INVALID), (dict(G=65536), INVALID), (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(T=1 << 31), INVALID), (dict(N=1 << 31, ldw=1 << 31, ldy=1 << 31), INVALID), (dict(K=1 << 31, ldx=1 << 31), INVALID),
    (dict(offsets=0), INVALID), (dict(offsets=PO + 2), UNSUPPORTED),
    (dict(ldx=31), INVALID), (dict(ldw=47), INVALID), (dict(ldy=47), INVALID), (dict(stride=-1), INVALID),
    (dict(ldx=1 << 60), INVALID), (dict(ldw=1 << 60), INVALID), (dict(stride=1 << 60), INVALID), (dict(stride=1 << 61), INVALID),
    (dict(X=0), INVALID), (dict(X=PX + 1), UNSUPPORTED),
])
def test_refusals(fn, kw, want):
    assert fn(**kw) == want, gemm.gemm_last_error()
    assert gemm.gemm_last_error() != ""


@pytest.mark.parametrize("kw, want", [
    (dict(trans=2), INVALID), (dict(trans=-1), INVALID), (dict(fill=2), INVALID), (dict(trans=1, ldw=31), INVALID),
    (dict(W=0), INVALID), (dict(Y=0), INVALID), (dict(Y=PY + 1), UNSUPPORTED), (dict(W=PW + 1), UNSUPPORTED),
    (dict(Y=PX), ALIAS), (dict(Y=PX + 2 * 64 * 32 - 2), ALIAS), (dict(Y=PW + 2 * (4 * 48 * 32 - 1)), ALIAS),
    (dict(Y=PO + 16), ALIAS), (dict(Y=PO - 63 * 96 - 96 + 4), ALIAS),
])
def test_refusals_of_the_product(kw, want):
    assert product(**kw) == want, gemm.gemm_last_error()
    assert gemm.gemm_last_error() != ""


@pytest.mark.parametrize("kw, want", [
    (dict(dW=0), INVALID), (dict(dY=0), INVALID), (dict(dW=PW + 2), UNSUPPORTED), (dict(dY=PY + 1), UNSUPPORTED),
    (dict(stride=0), INVALID), (dict(stride=48 * 32 - 1), INVALID), (dict(stride=48, ldw=4 * 48), INVALID),
    (dict(dW=PX), ALIAS), (dict(dW=PY), ALIAS), (dict(dW=PO + 16), ALIAS), (dict(dW=PX - 4 * (3 * 48 * 32 + 1)), ALIAS),
])
def test_refusals_of_the_gradient(kw, want):
    assert wgrad(**kw) == want, gemm.gemm_last_error()
    assert gemm.gemm_last_error() != ""


@pytest.mark.parametrize("kw", [dict(T=0, X=0, Y=0), dict(N=0, W=0, Y=0), dict(G=0, T=0, W=0, X=0, Y=0),
                                dict(G=0, W=0, fill=0)])
def test_empty_product_launches_nothing(kw):
    assert product(**kw) == OK, gemm.gemm_last_error()


@pytest.mark.parametrize("kw", [dict(G=0, dW=0), dict(N=0, dY=0, dW=0), dict(K=0, X=0, dW=0)])
def test_empty_gradient_launches_nothing(kw):
    assert wgrad(**kw) == OK, gemm.gemm_last_error()


@pytest.fixture(scope="module")
def bounds(tmp_path_factory):
    """grouped_bounds.h compiled for the host."""
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    folder = tmp_path_factory.mktemp("bounds")
    src = folder / "bounds.cc"
    src.write_text('''#include "grouped_bounds.h"
using namespace gemm::grouped;
extern "C" {
int h_clamp(int o, int T) { return clamp_offset(o, T); }
int h_runs(int i, int G, int fill) { return segment_runs(i, G, fill); }
int h_tiles(int rows, int bm) { return segment_tiles(rows, bm); }
int64_t h_most(int64_t T, int64_t G, int fill, int bm) { return most_tiles(T, G, fill, bm); }
}''')
    out = str(folder / "bounds.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(src), "-o", out], check=True)
    L = ctypes.CDLL(out)
    L.h_most.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    L.h_most.restype = ctypes.c_int64
    return L


def tiles_of(bounds, offsets, T, fill, bm):
    G = len(offsets) - 1
    ends, end = [], 0
    for i in range(G + 2):
        end = max(end, bounds.h_clamp(offsets[i], T)) if i <= G else T
        ends.append(end)
    starts = [0] + ends[:-1]
    assert ends[-1] == T and all(a <= b for a, b in zip(starts, ends))
    return sum(bounds.h_tiles(b - a, bm) for i, (a, b) in enumerate(zip(starts, ends)) if bounds.h_runs(i, G, fill))


@pytest.mark.parametrize("bm", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("fill", [0, 1])
def test_grid_holds_the_tiles_of_any_offsets(bounds, bm, fill):
    r = random.Random(bm + fill)
    for _ in range(300):
        G, T = r.choice([0, 1, 2, 5, 40]), r.choice([0, 1, 2, 3, bm - 1, bm, bm + 1, 1000])
        offsets = [r.randint(-3, T + 3) for _ in range(G + 1)]
        if r.random() < 0.7:
            offsets.sort()
        assert tiles_of(bounds, offsets, T, fill, bm) <= bounds.h_most(T, G, fill, bm)


@pytest.mark.parametrize("bm", [16, 64, 256])
def test_grid_is_no_larger_than_the_worst_offsets_need(bounds, bm):
    for G in (1, 3, 7):
        T = 5 * bm + 3 * G
        worst = [0] + [1 + bm * (i % 2) for i in range(G)]  # one row into a tile each
        offsets = [sum(worst[:i + 1]) for i in range(G + 1)]
        assert bounds.h_most(T, G, 0, bm) - tiles_of(bounds, offsets, offsets[-1], 0, bm) <= 6 + G
    assert bounds.h_most(2 ** 31 - 1, 65535, 1, bm) >= (2 ** 31 - 1) // bm


def test_rows_near_the_end_of_32_bits(bounds):
    top = 2 ** 31 - 1
    assert bounds.h_tiles(top, 256) == 2 ** 23 and bounds.h_tiles(top, 64) == 2 ** 25
    assert bounds.h_clamp(-2 ** 31, top) == 0 and bounds.h_clamp(top, top) == top and bounds.h_clamp(top, 5) == 5

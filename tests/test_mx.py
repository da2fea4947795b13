"""Microscaled operators on the host: exports, refusals before any launch,
the coded-matrix checks, and the oracle's own pins.  CPU only."""
import os
import re

import numpy as np
import pytest

from dense_gemm_row_amd import gemm, mx
from tests import mx_oracle as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PX, PQ, PS, PC = 0x10000000, 0x20000000, 0x30000000, 0x40000000  # never dereferenced
OK, INVALID, UNSUPPORTED, ALIAS = (gemm.GEMM_OK, gemm.GEMM_ERR_INVALID_ARG, gemm.GEMM_ERR_UNSUPPORTED,
                                   gemm.GEMM_ERR_ALIAS)


def test_exports_its_header():
    text = open(os.path.join(ROOT, "include", "gemm_mx.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(mx.EXPORTS)
    for n in names:
        assert hasattr(mx.lib(), n) and hasattr(mx, n)


def quant(dtype=2, fmt=0, trans=0, rows=4, cols=64, X=PX, ldx=64, codes=PQ, ldq=32, scales=PS, lds=2):
    return mx.gemm_mx_quantize(dtype, fmt, trans, rows, cols, X, ldx, codes, ldq, scales, lds)


def dequant(dtype=2, fmt=0, trans=0, rows=4, cols=64, X=PX, ldx=64, codes=PQ, ldq=32, scales=PS, lds=2):
    return mx.gemm_mx_dequantize(dtype, fmt, trans, rows, cols, codes, ldq, scales, lds, X, ldx)


@pytest.mark.parametrize("fn", [quant, dequant])
@pytest.mark.parametrize("kw, want", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID),
    (dict(trans=2), INVALID), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID),
    (dict(rows=1 << 31), INVALID), (dict(cols=1 << 31, ldx=1 << 31, ldq=1 << 30, lds=1 << 26), INVALID),
    (dict(ldx=63), INVALID), (dict(ldq=16), INVALID), (dict(ldq=31), INVALID), (dict(lds=1), INVALID),
    (dict(fmt=1, ldq=48), INVALID), (dict(cols=65, ldx=65), INVALID),
    (dict(trans=1, ldq=16, lds=0), INVALID),
    (dict(X=0), INVALID), (dict(codes=0), INVALID), (dict(scales=0), INVALID),
    (dict(ldx=1 << 62), INVALID), (dict(ldx=1 << 60), INVALID), (dict(ldq=1 << 62), INVALID),
    (dict(codes=PQ + 8), UNSUPPORTED), (dict(ldq=40), UNSUPPORTED), (dict(X=PX + 1), UNSUPPORTED),
    (dict(codes=PX), ALIAS), (dict(scales=PX + 3 * 128 + 127), ALIAS), (dict(codes=PX - 32 * 3 - 16), ALIAS),
])
def test_quantisation_refusals(fn, kw, want):
    assert fn(**kw) == want, gemm.gemm_last_error()
    assert gemm.gemm_last_error() != ""


def test_codes_and_scales_may_not_overlap():
    assert quant(scales=PQ + 16) == ALIAS


@pytest.mark.parametrize("kw", [dict(rows=0, X=0, codes=0, scales=0), dict(cols=0, X=0, codes=0, scales=0, ldq=0, lds=0)])
@pytest.mark.parametrize("fn", [quant, dequant])
def test_empty_quantisation_launches_nothing(fn, kw):
    assert fn(**kw) == OK
    assert gemm.gemm_last_error() == ""


def product(c=2, M=4, N=8, K=64, A=PX, lda=32, As=PX + 4096, ldas=2, B=PQ, ldb=32, Bs=PQ + 4096, ldbs=2, C=PC, ldc=8,
            epi=None):
    return mx.gemm_mx_matmul(c, M, N, K, A, lda, As, ldas, B, ldb, Bs, ldbs, C, ldc, None, epi)


@pytest.mark.parametrize("kw, want", [
    (dict(c=3), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(M=1 << 31), INVALID), (dict(N=1 << 31), INVALID), (dict(K=1 << 31), INVALID),
    (dict(lda=16), INVALID), (dict(ldb=16), INVALID), (dict(ldas=1), INVALID), (dict(ldbs=1), INVALID),
    (dict(ldc=7), INVALID), (dict(A=0), INVALID), (dict(As=0), INVALID), (dict(B=0), INVALID), (dict(Bs=0), INVALID),
    (dict(C=0), INVALID), (dict(epi=gemm.GemmEpilogue(1.0, 0.0, None, 5)), INVALID),
    (dict(A=PX + 4), UNSUPPORTED), (dict(B=PQ + 8), UNSUPPORTED), (dict(lda=40), UNSUPPORTED), (dict(C=PC + 1), UNSUPPORTED),
    (dict(epi=gemm.GemmEpilogue(1.0, 0.0, PC + 1024 + 2, 0)), UNSUPPORTED),
    (dict(C=PX), ALIAS), (dict(C=PX + 4096), ALIAS), (dict(C=PQ + 32), ALIAS), (dict(C=PQ + 4096), ALIAS),
    (dict(epi=gemm.GemmEpilogue(1.0, 0.0, PC + 16, 0)), ALIAS),
])
def test_product_refusals(kw, want):
    assert product(**kw) == want, gemm.gemm_last_error()
    assert gemm.gemm_last_error() != ""


def test_empty_product_launches_nothing():
    assert product(M=0, A=0, As=0, C=0) == OK
    assert product(N=0, B=0, Bs=0, C=0) == OK


def grad(y=2, c=0, T=64, F=4, N=8, codes=PX, ldq=64, scales=PX + 4096, lds=2, dY=PQ, ldy=8, dW=PC, ldw=8, ws=None,
         nws=0):
    return mx.gemm_mx_wgrad(y, c, T, F, N, codes, ldq, scales, lds, dY, ldy, dW, ldw, 1.0, 0.0, ws, nws)


@pytest.mark.parametrize("kw, want", [
    (dict(y=3), INVALID), (dict(c=4), INVALID), (dict(T=-1), INVALID), (dict(F=-1), INVALID), (dict(N=-1), INVALID),
    (dict(T=1 << 31), INVALID), (dict(ldq=32), INVALID), (dict(lds=1), INVALID), (dict(ldy=7), INVALID),
    (dict(ldw=7), INVALID), (dict(codes=0), INVALID), (dict(scales=0), INVALID), (dict(dY=0), INVALID),
    (dict(dW=0), INVALID), (dict(nws=-1), INVALID),
    (dict(codes=PX + 8), UNSUPPORTED), (dict(ldq=72), UNSUPPORTED), (dict(dY=PQ + 1), UNSUPPORTED),
    (dict(dW=PC + 2), UNSUPPORTED),
    (dict(dW=PX), ALIAS), (dict(dW=PX + 4096), ALIAS), (dict(dW=PQ), ALIAS),
])
def test_gradient_refusals(kw, want):
    assert grad(**kw) == want, gemm.gemm_last_error()
    assert gemm.gemm_last_error() != ""


def test_gradient_workspace_checks():
    assert mx.gemm_mx_wgrad_workspace_bytes(3, 1, 1, 1) == -1
    assert mx.gemm_mx_wgrad_workspace_bytes(2, -1, 1, 1) == -1
    assert mx.gemm_mx_wgrad_workspace_bytes(2, 1, 1 << 31, 1) == -1
    assert mx.gemm_mx_wgrad_workspace_bytes(2, 32, 4096, 4096) == 0
    for big in [(2, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (0, 2 ** 31 - 1, 1, 1), (1, 1, 2 ** 31 - 1, 1)]:
        assert mx.gemm_mx_wgrad_workspace_bytes(*big) >= 0


def test_coded_matrix_checks():
    import torch
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    q = mx.MxTensor(u8(3, 32), u8(3, 2), 64)
    assert q.shape == (3, 64) and q.nbytes() == 3 * 34
    mx.MxTensor(u8(3, 32), u8(3, 2), 33)
    mx.MxTensor(u8(3, 64), u8(3, 4)[:, :2], 64, mx.E4M3)
    for bad in [lambda: mx.MxTensor(u8(3, 32), u8(3, 2), 65), lambda: mx.MxTensor(u8(3, 32), u8(3, 2), 32),
                lambda: mx.MxTensor(u8(3, 32), u8(2, 2), 64), lambda: mx.MxTensor(u8(3, 32), u8(3, 2), 64, "e5m2"),
                lambda: mx.MxTensor(u8(32, 3).t(), u8(3, 2), 64), lambda: mx.MxTensor(u8(96), u8(3, 2), 64),
                lambda: mx.MxTensor(u8(3, 32).float(), u8(3, 2), 64)]:
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        mx.empty(2, 2, "e5m2", "cpu")


def test_torch_forms_refuse_what_they_do_not_take():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = mx.empty(4, 64, mx.E2M1, "cpu")
    with pytest.raises(ValueError):
        mx.quantize(x)  # not on the GPU
    with pytest.raises(TypeError):
        mx.quantize(x.to(torch.float64))
    with pytest.raises(ValueError):
        mx.quantize(x[0])
    with pytest.raises(ValueError):
        mx.quantize(x.t())
    with pytest.raises(ValueError):
        mx.dequantize(q)
    with pytest.raises(TypeError):
        mx.dequantize(x)
    with pytest.raises(TypeError):
        mx.matmul(x, x)
    with pytest.raises(ValueError):
        mx.matmul(x, q)
    with pytest.raises(ValueError):
        mx.weight_grad(q, x)  # 4-bit codes
    with pytest.raises(ValueError):
        mx.restore(q)


# -- the oracle -------------------------------------------------------------
def test_oracle_pins():
    # 1 .. 6 of amax 6: scale 1; midpoints go to the even code.
    row = np.zeros((1, 32))
    row[0, :10] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -5]
    c, s = oracle.quantize(row, "e2m1")
    assert s[0, 0] == 127 and list(c[0, 0, :10]) == [7, 6, 6, 4, 4, 2, 2, 0, 8, 14]
    # amax 7.9: the OCP rule keeps exponent 0 and saturates.
    row[0, 0] = 7.9
    c, s = oracle.quantize(row, "e2m1")
    assert s[0, 0] == 127 and c[0, 0, 0] == 7
    # E4M3: 448 keeps exponent 0, one ulp more takes the next.
    row[0, 0] = 448
    assert oracle.quantize(row, "e4m3")[1][0, 0] == 127
    row[0, 0] = np.nextafter(448, 449)
    assert oracle.quantize(row, "e4m3")[1][0, 0] == 128
    row[0, 0] = 256
    assert oracle.quantize(row, "e4m3")[1][0, 0] == 127
    row[:] = 0
    assert oracle.quantize(row, "e4m3")[1][0, 0] == 0
    row[0, 3] = np.inf
    c, s = oracle.quantize(row, "e2m1")
    assert s[0, 0] == 255 and not c.any()


@pytest.mark.parametrize("fmt, step", [("e2m1", 2.0 ** -2), ("e4m3", 2.0 ** -4)])
def test_oracle_error_bounds(fmt, step):
    """Half a step of each element's binade, or of the block's smallest; a
    saturated E2M1 element loses up to a quarter (8 to 6)."""
    x = np.random.default_rng(3).standard_normal((64, 100)) * np.exp(np.random.default_rng(4).uniform(-9, 9, (64, 1)))
    got = oracle.round_trip(x, fmt)
    small = {"e2m1": 0.25, "e4m3": 2.0 ** -10}[fmt]
    s = np.ldexp(1.0, oracle.quantize(x, fmt)[1].astype(int) - 127)
    floor = np.repeat(s, 32, axis=1)[:, :100] * small
    assert np.all(np.abs(got - x) <= np.maximum(step * np.abs(x), floor))

"""4-bit weights with group scales on the host: exports, refusals before any
launch, the coded-weight checks, and the oracle's own pins.  CPU only."""
import fractions
import os
import re

import numpy as np
import pytest

from dense_gemm_row_amd import gemm, w4
from tests import w4_oracle as oracle

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PX, PQ, PS, PZ, PY, PO, PK = (i << 28 for i in range(1, 8))  # never dereferenced
OK, INVALID, UNSUPPORTED, ALIAS = (gemm.GEMM_OK, gemm.GEMM_ERR_INVALID_ARG, gemm.GEMM_ERR_UNSUPPORTED,
                                   gemm.GEMM_ERR_ALIAS)
F32, F16, BF16 = gemm.DTYPE_F32, gemm.DTYPE_F16, gemm.DTYPE_BF16


def test_exports_its_header():
    text = open(os.path.join(ROOT, "include", "gemm_w4.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(w4.EXPORTS)
    for n in names:
        assert hasattr(w4.lib(), n) and hasattr(w4, n)
    assert int(re.search(r"#define GEMM_W4_ROWS (\d+)", text).group(1)) == w4.ROWS


def desc(codes=PQ, ldq=64, stride_q=64 * 48, scales=PS, lds=1, stride_s=48, zeros=PZ, ldz=1, stride_z=48, group=128):
    return w4.GemmW4(codes, ldq, stride_q, scales, lds, stride_s, zeros or None, ldz, stride_z, group)


def split(kw):
    mine = {k: kw.pop(k) for k in list(kw) if k in w4.GemmW4.__dict__ and k != "group"}
    if "group" in kw:
        mine["group"] = kw.pop("group")
    return desc(**mine)


def quant(dtype=BF16, s_dtype=BF16, trans=0, N=48, K=128, X=PX, ldx=128, q=None, **kw):
    return w4.gemm_w4_quantize(dtype, s_dtype, trans, N, K, X, ldx, q or split(kw))


def dequant(dtype=BF16, s_dtype=BF16, N=48, K=128, X=PX, ldx=128, q=None, **kw):
    return w4.gemm_w4_dequantize(dtype, s_dtype, N, K, q or split(kw), X, ldx)


def product(dtype=BF16, M=4, N=48, K=128, X=PX, ldx=128, Y=PY, ldy=48, ws=0, wb=0, q=None, **kw):
    return w4.gemm_w4_matmul(dtype, M, N, K, X, ldx, q or split(kw), Y, ldy, ws, wb)


def experts(dtype=BF16, G=3, T=4, N=48, K=128, offsets=PO, X=PX, ldx=128, Y=PY, ldy=48, fill=1, ws=0, wb=0, q=None, **kw):
    return w4.gemm_w4_grouped(dtype, G, T, N, K, offsets, X, ldx, q or split(kw), Y, ldy, fill, ws, wb)


@pytest.mark.parametrize("fn", [quant, dequant, product, experts])
@pytest.mark.parametrize("kw, want", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(group=16), INVALID), (dict(group=0), INVALID),
    (dict(group=256), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(N=1 << 31, ldy=1 << 31), INVALID),
    (dict(K=(1 << 30) + 1, ldx=1 << 31, ldq=1 << 30, lds=1 << 25, ldz=1 << 25), INVALID),
    (dict(ldx=127), INVALID), (dict(ldq=63), INVALID), (dict(ldq=48), INVALID), (dict(lds=0), INVALID), (dict(ldz=0), INVALID),
    (dict(group=64), INVALID),  # two groups a row: lds and ldz are 1
    (dict(X=0), INVALID), (dict(codes=0), INVALID), (dict(scales=0), INVALID),
    (dict(ldx=1 << 60), INVALID), (dict(ldq=1 << 60), INVALID), (dict(lds=1 << 60), INVALID), (dict(ldz=1 << 62), INVALID),
    (dict(codes=PQ + 8), UNSUPPORTED), (dict(ldq=72), UNSUPPORTED), (dict(X=PX + 1), UNSUPPORTED), (dict(scales=PS + 1), UNSUPPORTED),
])
def test_refusals(fn, kw, want):
    assert fn(**dict(kw)) == want, gemm.gemm_last_error()
    assert gemm.gemm_last_error() != ""


def test_a_missing_description_is_refused():
    L = w4.lib()
    assert L.gemm_w4_quantize(BF16, BF16, 0, 4, 32, PX, 32, None, None) == INVALID
    assert L.gemm_w4_dequantize(BF16, BF16, 4, 32, None, PX, 32, None) == INVALID
    assert L.gemm_w4_matmul(BF16, 1, 4, 32, PX, 32, None, PY, 4, None, 0, None) == INVALID
    assert L.gemm_w4_grouped(BF16, 2, 1, 4, 32, PO, PX, 32, None, PY, 4, 1, None, 0, None) == INVALID


@pytest.mark.parametrize("kw, want", [
    (dict(s_dtype=F32), INVALID), (dict(trans=2), INVALID), (dict(trans=1, ldx=47), INVALID), (dict(dtype=F32, X=PX + 2), UNSUPPORTED),
    (dict(codes=PX), ALIAS), (dict(scales=PX + 2), ALIAS), (dict(zeros=PX + 1), ALIAS), (dict(scales=PQ), ALIAS),
    (dict(zeros=PQ + 1), ALIAS), (dict(zeros=PS), ALIAS),
])
def test_refusals_of_quantisation(kw, want):
    assert quant(**dict(kw)) == want, gemm.gemm_last_error()


@pytest.mark.parametrize("kw, want", [(dict(s_dtype=F32), INVALID), (dict(X=PQ), ALIAS), (dict(X=PS), ALIAS), (dict(X=PZ), ALIAS)])
def test_refusals_of_dequantisation(kw, want):
    assert dequant(**dict(kw)) == want, gemm.gemm_last_error()


NEED = 2 * 48 * 128


@pytest.mark.parametrize("fn, many, scale", [(product, dict(M=129), 1), (experts, dict(T=385), 3)])
@pytest.mark.parametrize("kw, want", [
    (dict(dtype=F32), INVALID), (dict(ldy=47), INVALID), (dict(Y=0), INVALID), (dict(Y=PY + 1), UNSUPPORTED),
    (dict(Y=PX), ALIAS), (dict(Y=PQ), ALIAS), (dict(Y=PS), ALIAS), (dict(Y=PZ), ALIAS), (dict(wb=-1), INVALID),
    (dict(many=1), INVALID), (dict(many=1, ws=PK, wb=-1), INVALID), (dict(many=1, ws=PK, wb=NEED - 1), INVALID),
    (dict(many=1, ws=0, wb=1 << 30), INVALID), (dict(many=1, ws=PK + 8, wb=1 << 30), INVALID),
    (dict(many=1, ws=PX, wb=1 << 20), ALIAS), (dict(many=1, ws=PQ, wb=1 << 20), ALIAS), (dict(many=1, ws=PY, wb=1 << 20), ALIAS),
])
def test_refusals_of_the_products(fn, many, scale, kw, want):
    kw = dict(kw)
    if kw.pop("many", 0):
        kw.update(many)
    if kw.get("wb") == NEED - 1:
        kw["wb"] = scale * NEED - 1
    assert fn(**kw) == want, gemm.gemm_last_error()


@pytest.mark.parametrize("kw, want", [
    (dict(G=-1), INVALID), (dict(G=65536), INVALID), (dict(T=-1), INVALID), (dict(fill=2), INVALID), (dict(offsets=0), INVALID),
    (dict(offsets=PO + 2), UNSUPPORTED), (dict(Y=PO), ALIAS), (dict(stride_q=-16), INVALID), (dict(stride_q=8), UNSUPPORTED),
    (dict(stride_s=-1), INVALID), (dict(stride_z=-1), INVALID), (dict(stride_q=1 << 62), INVALID), (dict(Y=PQ + 2 * 64 * 48), ALIAS),
])
def test_refusals_of_the_grouped_product(kw, want):
    assert experts(**dict(kw)) == want, gemm.gemm_last_error()


def test_empty_calls_launch_nothing():
    assert quant(N=0, X=0, codes=0, scales=0) == OK and quant(K=0, X=0, codes=0, scales=0, zeros=0) == OK
    assert dequant(N=0) == OK and dequant(K=0) == OK
    assert product(M=0, X=0, Y=0) == OK and product(N=0, codes=0, scales=0, Y=0) == OK
    assert experts(T=0, X=0, Y=0) == OK and experts(N=0, codes=0, scales=0, Y=0) == OK
    assert experts(G=0, codes=0, scales=0, fill=0) == OK


def test_workspace_sizes():
    for M, N, K in ((0, 5, 64), (1, 48, 128), (128, 48, 128), (129, 48, 0)):
        assert w4.gemm_w4_matmul_workspace_bytes(M, N, K) == 0
    assert w4.gemm_w4_matmul_workspace_bytes(129, 48, 128) == NEED
    assert w4.gemm_w4_matmul_workspace_bytes(129, 48, 121) == NEED
    assert w4.gemm_w4_grouped_workspace_bytes(3, 384, 48, 128) == 0
    assert w4.gemm_w4_grouped_workspace_bytes(3, 385, 48, 128) == 3 * NEED
    assert w4.gemm_w4_grouped_workspace_bytes(0, 5, 48, 128) == 0
    top = 2 ** 31 - 1
    assert w4.gemm_w4_matmul_workspace_bytes(129, top, 2 ** 30) == 2 * top * 2 ** 30
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (2 ** 31, 1, 1), (1, 1, 2 ** 30 + 1)):
        assert w4.gemm_w4_matmul_workspace_bytes(*bad) == -1
    for bad in ((-1, 1, 1, 1), (65536, 1, 1, 1), (1, 2 ** 31, 1, 1), (65535, 2 ** 31 - 1, top, 2 ** 30)):
        assert w4.gemm_w4_grouped_workspace_bytes(*bad) == -1


def test_coded_weights_are_checked():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    q = w4.W4Tensor(u8(6, 64), bf(6, 1), u8(6, 1), 128)
    assert q.shape == (6, 128) and q.nbytes() == 6 * 64 + 12 + 6
    stack = w4.W4Tensor(u8(3, 6, 64), bf(3, 6, 4), None, 100, 32)
    assert stack.shape == (3, 6, 100) and stack[1].shape == (6, 100)
    for error, make in [
        (ValueError, lambda: w4.W4Tensor(u8(6, 64), bf(6, 1), None, 128, 16)),
        (ValueError, lambda: w4.W4Tensor(u8(6, 64), bf(6, 1), None, 129)),
        (ValueError, lambda: w4.W4Tensor(u8(6, 64), bf(6, 2), None, 128)),
        (ValueError, lambda: w4.W4Tensor(u8(6, 64), bf(5, 1), None, 128)),
        (ValueError, lambda: w4.W4Tensor(u8(6, 64), bf(6, 1), u8(6, 2), 128)),
        (ValueError, lambda: w4.W4Tensor(u8(64), bf(1), None, 128)),
        (ValueError, lambda: w4.W4Tensor(u8(6, 64).to(torch.int8), bf(6, 1), None, 128)),
        (TypeError, lambda: w4.W4Tensor(u8(6, 64), bf(6, 1).float(), None, 128)),
        (TypeError, lambda: w4.W4Tensor(u8(6, 64), bf(6, 1), bf(6, 1), 128)),
        (ValueError, lambda: w4.W4Tensor(u8(6, 128)[:, ::2], bf(6, 1), None, 128)),
        (ValueError, lambda: w4.W4Tensor(u8(64, 6).t(), bf(6, 1), None, 128)),
        (TypeError, lambda: q[0]),
        (ValueError, lambda: w4.matmul(bf(1, 128), q)),        # not on the GPU
        (TypeError, lambda: w4.matmul(bf(1, 128), bf(6, 128))),
        (ValueError, lambda: w4.quantize(bf(6, 128))),
        (ValueError, lambda: w4.dequantize(q)),
    ]:
        with pytest.raises(error):
            make()


# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------
def test_oracle_rounds_ratios_as_rationals_do():
    r = np.random.default_rng(1)
    for kind in ("f16", "bf16"):
        s = oracle.rounded(np.exp(r.uniform(-9, 3, 400)).astype(np.float32), kind)
        t = r.integers(-16, 17, 400) + r.choice([0, 0.5, 0.25], 400)
        near = (t * s).astype(np.float32)
        for w in (near, np.nextafter(near, np.float32(np.inf)), np.nextafter(near, np.float32(-np.inf))):
            want = [round(fractions.Fraction(float(a)) / fractions.Fraction(float(b))) for a, b in zip(w, s)]
            assert np.array_equal(oracle.nearest(w.astype(np.float64), s), want)


def test_oracle_packs_and_decodes():
    codes = np.arange(40, dtype=np.uint8).reshape(1, 40) % 16
    packed = oracle.pack(codes)
    assert packed.shape == (1, 32) and packed[0, 0] == 0x10 and packed[0, 19] == 0x76 and packed[0, 20] == 0
    assert np.array_equal(oracle.unpack(packed, 40), codes)
    v, size = oracle.values(codes, np.array([[2.0, 0.5]]), np.array([[8, 3]], np.uint8), 32)
    assert v[0, 0] == -16 and v[0, 31] == 14 and v[0, 32] == -1.5 and size[0, 31] == 110 and size[0, 39] == 21


def test_oracle_quantises_by_hand():
    w = np.zeros((3, 64))
    w[0, :3] = [-3.0, 12.0, 4.5]   # span 15: scale 1, zero point 3; 4.5 is a tie between 4 and 5
    w[1, :3] = [7.0, -7.0, 2.5]    # largest 7: scale 1; 2.5 is a tie between 2 and 3
    w[2, 40] = np.inf
    q, s, z = oracle.quantize(w, 32, True, "bf16")
    assert s[0, 0] == 1 and z[0, 0] == 3 and list(q[0, :4]) == [0, 15, 7, 3]
    assert s[0, 1] == 0 and z[0, 1] == 0 and not q[0, 32:].any()
    assert s[2, 0] == 0 and np.isnan(s[2, 1]) and z[2, 1] == 0 and not q[2, 32:].any()
    q, s, z = oracle.quantize(w, 32, False, "f16")
    assert s[1, 0] == 1 and list(q[1, :4]) == [15, 1, 10, 8] and (q[1, 32:] == 8).all() and (z[:2] == 8).all()

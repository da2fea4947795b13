"""The pipelined kernels' tiles against 64 bits: scale rows of whole 4 and 16
bytes with NaN bytes (255) behind the matrix' blocks, k that ends anywhere in
the four slices of the loop, both tile sizes, with and without the epilogue.

Bounds as in test_gpu_mx: exact sums bit for bit, general values within
(n + 8) * 2^-23 of sum|a b| plus the type's half step."""
import numpy as np
import pytest

from dense_gemm_row_amd import gemm, mx
from tests import mx_oracle as oracle
from tests.mx_sizes import LARGE_GRADS, LARGE_PRODUCTS
from tests.test_gpu_mx import TYPES, dense, near, rng, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def scale_rows(scales, unit):
    """The scale bytes in rows of a multiple of `unit` bytes (4: and not of
    16), 255 behind them."""
    rows, nb = scales.shape
    width = -(-nb // unit) * unit
    if unit == 4 and width % 16 == 0:
        width += 4
    whole = torch.full((rows, width), 255, dtype=torch.uint8, device="cuda")
    whole[:, :nb] = torch.from_numpy(scales)
    return whole[:, :nb]


def coded(r, rows, cols, lo, hi, unit, fmt=mx.E2M1):
    """Random codes and scale bytes in [lo, hi); (MxTensor, values)."""
    nb = -(-cols // 32)
    elem = r.integers(0, 16, (rows, nb * 32)).astype(np.uint8)
    elem[:, cols:] = 0
    packed, scales = oracle.pack(elem, fmt), r.integers(lo, hi, (rows, nb)).astype(np.uint8)
    q = mx.MxTensor(torch.from_numpy(packed).cuda(), scale_rows(scales, unit), cols, fmt)
    return q, oracle.values(packed, scales, cols, fmt)


KS = [1, 33, 257, 1000, 1056, 2090, 4097, 4608]  # 1 to 18 slices of 256, odd and even blocks


@pytest.mark.parametrize("unit", [4, 16])
@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("m", [17, 130])
def test_product(m, k, unit):
    r = rng(m, k, unit, 41)
    n = 131
    a, av = coded(r, m, k, 110, 131, unit)
    b, bv = coded(r, n, k, 110, 131, unit)
    want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
    for out in TYPES:
        got = mx.matmul(a, b, out_dtype=TYPES[out]).double().cpu().numpy()
        keep = size < 6e4  # in binary16's range
        assert np.all(near(got, want, size, k, out)[keep])
    # Exact sums through the epilogue.
    a, av = coded(r, m, k, 126, 128, unit)
    b, bv = coded(r, n, k, 126, 128, unit)
    bias = torch.from_numpy(r.integers(-64, 64, n) / 4.0).float().cuda()
    for out in TYPES:
        old, oldv = dense(r.integers(-32, 32, (m, n)) / 2.0, out)
        exact = 0.5 * (av @ bv.T) + 2.0 * oldv + bias.double().cpu().numpy()
        mx.matmul(a, b, out=old, alpha=0.5, beta=2.0, bias=bias, act=gemm.ACT_RELU)
        assert torch.equal(old.cpu(), torch.from_numpy(np.maximum(exact, 0.0)).to(TYPES[out]))


@pytest.mark.parametrize("unit", [4, 16])
@pytest.mark.parametrize("k", [33, 1000, 4097])
def test_product_with_nan_blocks(k, unit):
    """First and last block of a row: its results are NaN, no others."""
    r = rng(k, unit, 42)
    a, _ = coded(r, 130, k, 126, 128, unit)
    b, _ = coded(r, 131, k, 126, 128, unit)
    a.scales[5, 0] = a.scales[129, -1] = b.scales[130, 0] = b.scales[64, -1] = 255
    want = np.zeros((130, 131), bool)
    want[[5, 129]] = True
    want[:, [130, 64]] = True
    assert np.array_equal(torch.isnan(mx.matmul(a, b)).cpu().numpy(), want)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m", [17, 130])
@pytest.mark.parametrize("k", [33, 1000, 4097])
def test_product_of_many_values(m, k, kind):
    r = rng(m, k, 43)
    x, exact = dense(values(r, m, k).clip(-1e3, 1e3), kind)
    b, bv = coded(r, 131, k, 120, 126, 4)
    av = oracle.round_trip(exact, "e2m1")
    got = mx.matmul(x, b, out_dtype=torch.float32).double().cpu().numpy()
    assert np.all(near(got, av @ bv.T, np.abs(av) @ np.abs(bv).T, k, "f32"))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m", [1, 5, 16])
@pytest.mark.parametrize("k", [4, 100, 516, 4100, 4608])
def test_few_aligned_values_give_the_bits_of_their_codes(m, k, kind):
    """With rows on 16 bytes and scales on whole words both ways add in one
    order."""
    r = rng(m, k, 44)
    x, _ = dense(values(r, m, k).clip(-1e3, 1e3), kind, pad=-k % 8)
    b, _ = coded(r, 37, k, 120, 126, 4)
    for out in TYPES:
        assert torch.equal(mx.matmul(x, b, out_dtype=TYPES[out]), mx.matmul(mx.quantize(x), b, out_dtype=TYPES[out]))


@pytest.mark.parametrize("unit", [4, 16])
@pytest.mark.parametrize("m, n, k", LARGE_PRODUCTS)
def test_product_on_large_tiles(m, n, k, unit):
    """Exact sums (multiples of 1/16 below 36 * k < 2^20), so the 64-bit
    product of the same values is the result before its rounding."""
    r = rng(m, n, k, 45)
    a, av = coded(r, m, k, 126, 128, unit)
    b, bv = coded(r, n, k, 126, 128, unit)
    exact = torch.from_numpy(av).cuda() @ torch.from_numpy(bv).cuda().t().contiguous()
    bias = torch.from_numpy(r.integers(-64, 64, n) / 4.0).float().cuda()
    old = torch.from_numpy(r.integers(-32, 32, (m, n)) / 2.0).cuda()
    for kind in TYPES:
        t = TYPES[kind]
        for pad in (0, 3):
            c = torch.full((m, n + pad), 7.0, dtype=t, device="cuda")
            mx.matmul(a, b, out=c[:, :n])
            assert torch.equal(c[:, :n], exact.to(t)) and bool((c[:, n:] == 7.0).all())
            c[:, :n] = old
            mx.matmul(a, b, out=c[:, :n], alpha=0.5, beta=2.0, bias=bias, act=gemm.ACT_RELU)
            assert torch.equal(c[:, :n], (0.5 * exact + 2.0 * old + bias.double()).clamp(min=0.0).to(t))
            assert bool((c[:, n:] == 7.0).all())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t, f, n", LARGE_GRADS)
def test_gradient_on_large_tiles(t, f, n, kind):
    """Integers of |x| <= 8 (exact in E4M3) and |dy| <= 8: sums below 2^24."""
    r = rng(t, f, n, 46)
    x = torch.from_numpy(r.integers(-8, 9, (t, f)).astype(np.float64)).cuda()
    dy = torch.from_numpy(r.integers(-8, 9, (t, n)).astype(np.float64)).cuda()
    q = mx.checkpoint(x.to(torch.bfloat16))
    kept = mx.MxTensor(q.codes, scale_rows(q.scales.cpu().numpy(), 4), t, mx.E4M3)
    exact = x.t().contiguous() @ dy
    old = torch.from_numpy(r.integers(-32, 32, (f, n)).astype(np.float64)).cuda()
    for out in TYPES:
        o = TYPES[out]
        c = torch.full((f, n + 3), 7.0, dtype=o, device="cuda")
        mx.weight_grad(kept, dy.to(TYPES[kind]), out=c[:, :n])
        assert torch.equal(c[:, :n], exact.to(o)) and bool((c[:, n:] == 7.0).all())
        c = old.to(o)
        mx.weight_grad(kept, dy.to(TYPES[kind]), out=c, alpha=2.0, beta=-1.0)
        assert torch.equal(c, (2.0 * exact - old).to(o))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("t, f, n", [(20, 40, 24), (300, 136, 72)])
def test_gradient_of_tiny_values(t, f, n, kind):
    """dY far below 2^-110, where its lower bfloat16 terms are subnormal, with
    activations that bring the sums back to ordinary size.  A term keeps
    multiples of 2^-133, so each dY is off by less than that."""
    r = rng(t, f, n, 47)
    x, _ = dense(r.standard_normal((t, f)) * 2.0 ** 90, "f32")
    kept = mx.checkpoint(x)
    xv = oracle.values(kept.codes.cpu().numpy(), kept.scales.cpu().numpy(), t, "e4m3")
    dy, dyv = dense(r.standard_normal((t, n)) * 2.0 ** -118, kind)
    got = mx.weight_grad(kept, dy).double().cpu().numpy()
    want, size = xv @ dyv, np.abs(xv) @ np.abs(dyv)
    lost = np.abs(xv).sum(1, keepdims=True) * 2.0 ** -133
    assert np.all(np.abs(got - want) <= (3 * t + 8) * 2.0 ** -23 * size + lost)


@pytest.mark.parametrize("unit", [1, 4, 16])
@pytest.mark.parametrize("m", [5, 40, 130])
def test_product_of_the_scales_ends(m, unit):
    """Factors down to 2^-127 times factors up to 2^127: multiples of 2^-5
    below 2^16, exact in FP32."""
    r = rng(m, unit, 48)
    a, av = coded(r, m, 257, 0, 3, unit)
    b, bv = coded(r, 70, 257, 252, 255, unit)
    exact = torch.from_numpy(av @ bv.T)
    assert torch.equal(mx.matmul(a, b, out_dtype=torch.float32).cpu(), exact.float())
    assert torch.equal(mx.matmul(b, a, out_dtype=torch.float32).cpu(), exact.t().float())

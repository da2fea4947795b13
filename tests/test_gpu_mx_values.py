"""Products of values on the GPU: every way of taking them gives what
quantising first gives, bit for bit, at row counts around a decoding step's 16
and with rows, scales and strides off the fast layout."""
import numpy as np
import pytest

from dense_gemm_row_amd import mx
from tests.test_gpu_mx import TYPES, dense, random_coded, rng, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m", [1, 3, 9, 16, 17, 130])
@pytest.mark.parametrize("k", [1, 31, 100, 512, 1056, 4097, 4608])
def test_values_are_quantise_then_product(m, k, kind):
    r = rng(m, k, 21)
    v = values(r, m, k).clip(-1e3, 1e3)
    w, _ = random_coded(r, 37, k, mx.E2M1, 120, 126, pad=1)
    aligned = mx.empty(37, k, mx.E2M1, "cuda")  # scale rows of whole words
    aligned.codes.copy_(w.codes)
    aligned.scales.copy_(w.scales)
    for pad, shift in ((0, 0), (-k % 16, 0), (-k % 16 + 16, 0), (1, 0), (-k % 16, 1)):
        x, _ = dense(v, kind, pad, shift)
        for b in (w, aligned):
            got = mx.matmul(x, b, out_dtype=torch.float32)
            want = mx.matmul(mx.quantize(x.contiguous()), b, out_dtype=torch.float32)
            if m <= 16:
                # Up to 16 rows the sums' order depends on the layout: any
                # two orders of k FP32 additions are this close.
                size = mx.matmul(mx.MxTensor(mx.quantize(x.contiguous()).codes & 0x77, mx.quantize(x.contiguous()).scales, k),
                                 mx.MxTensor(b.codes & 0x77, b.scales, k), out_dtype=torch.float32)
                assert bool(((got - want).abs() <= 2 * (k + 8) * 2.0 ** -23 * size).all())
            else:
                assert torch.equal(got, want)


@pytest.mark.parametrize("kind", TYPES)
def test_values_with_infinities(kind):
    """An infinity or NaN makes its block, and so its row, NaN; no other."""
    r = rng(22)
    v = r.standard_normal((16, 300))
    v[3, 299] = np.inf
    v[7, 40] = np.nan
    x, _ = dense(v, kind, pad=4)
    w, _ = random_coded(r, 50, 300, mx.E2M1, 126, 128)
    bad = torch.isnan(mx.matmul(x, w, out_dtype=torch.float32)).all(dim=1).cpu().numpy()
    assert list(np.nonzero(bad)[0]) == [3, 7]
    assert not torch.isnan(mx.matmul(x, w, out_dtype=torch.float32)).any(dim=1).cpu().numpy()[[0, 4, 15]].any()


def test_far_rows():
    """Rows of X and of the weights' codes past 2^31 bytes of their buffer."""
    big = torch.empty(5 << 30, dtype=torch.uint8, device="cuda")
    r = rng(23)
    x = big.view(torch.bfloat16)[: (5 << 29)].view(5, 1 << 29)[:, :96]
    x.copy_(torch.from_numpy(r.standard_normal((5, 96))))
    w, _ = random_coded(r, 20, 96, mx.E2M1, 126, 128)
    assert torch.equal(mx.matmul(x, w), mx.matmul(x.contiguous(), w))
    near = mx.quantize(torch.from_numpy(r.standard_normal((3, 96))).float().cuda())
    far = mx.MxTensor(big.view(5 << 10, 1 << 20)[1::2048][:3, :48], near.scales, 96)
    far.codes.copy_(near.codes)
    y = torch.from_numpy(r.standard_normal((4, 96))).to(torch.bfloat16).cuda()
    assert torch.equal(mx.matmul(y, far), mx.matmul(y, near))


@pytest.mark.parametrize("m", [2, 40])
def test_values_graph_and_streams(m):
    r = rng(24, m)
    x = torch.zeros(m, 520, dtype=torch.bfloat16, device="cuda")
    w, _ = random_coded(r, 72, 520, mx.E2M1, 126, 128)
    mx.matmul(x, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mx.matmul(x, w)
    s = torch.cuda.Stream()
    for k in range(4):
        x.copy_(torch.from_numpy(r.standard_normal((m, 520))))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx.matmul(x, w)), k
        other = mx.matmul(x, w, stream=s)
        s.synchronize()
        assert torch.equal(out, other)

"""4-bit products of activations that are infinite, NaN, or so large that the
kernels' sums of (16 + q) x leave FP32: the results are those of the
definition, y = sum of s (q - z) x, in every kernel, with few rows and with
many.  Other rows' results stay exact."""
import numpy as np
import pytest

from dense_gemm_row_amd import w4
from tests.test_gpu_w4 import SCALES, TYPES, coded, dense, gpu, rng, whole

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def product(x, w):
    """Row by column in 64 bits, infinities and NaN as they come."""
    with np.errstate(invalid="ignore"):
        return np.array([(row * w).sum(axis=1) for row in x]).reshape(len(x), len(w))


def same(got, exact, kind):
    want = torch.from_numpy(exact).to(TYPES[kind])
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(nan=0.0, posinf=np.inf, neginf=-np.inf), want.nan_to_num(nan=0.0, posinf=np.inf, neginf=-np.inf))


def special(x, kind, K):
    """Rows of infinities and NaN in the first and last groups; in bfloat16 also
    2^124, 16 of which leave FP32 (one a row, or with its negative: with scales
    of 2^-6 and whole codes every sum of the definition is exact)."""
    x[0, K // 2] = np.inf
    if len(x) < 8:
        return x
    x[1, 0], x[2, K - 1] = -np.inf, np.inf
    x[3, 0] = x[3, K - 1] = np.inf
    x[4, 0], x[4, K - 1] = np.inf, -np.inf
    x[5, K // 3] = np.nan
    if kind == "bf16":
        x[6], x[7] = 0, 0
        x[6, K // 2] = 2.0 ** 124
        x[7, 0], x[7, K - 1] = -2.0 ** 124, 2.0 ** 124
    return x


# Few rows of one to four blocks of 16, in whole spans, in spans that end inside
# and by element, and many rows.
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("N, K", [(40, 512), (72, 300), (17, 31), (136, 2048)])
def test_infinite_and_large_activations(N, K, kind, group, zeros):
    r = rng(11, N, K, group)
    q, value, _ = coded(r, (N, K), group, kind, zeros, -6, -5, whole=True)
    for M in (1, 16, 33, 64, 128, 129):
        x, ex = dense(special(64.0 * whole(r, (M, K)), kind, K), kind)
        same(w4.matmul(x, q), product(ex, value), kind)


@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("T, G", [(60, 3), (400, 3)])
@pytest.mark.parametrize("K", [512, 300])
def test_infinite_and_large_activations_of_experts(K, T, G, kind, group):
    r = rng(12, K, T, group)
    q, value, _ = coded(r, (G, 40, K), group, kind, True, -6, -5, whole=True)
    x, ex = dense(64.0 * whole(r, (T, K)), kind)
    bounds = [2, 30, 30, T - 3]
    ex[:2] = np.nan
    ex[2:12] = special(ex[2:12], kind, K)
    ex[30:40] = special(ex[30:40], kind, K)
    ex[T - 3:] = np.inf
    x.copy_(torch.from_numpy(ex))
    exact = np.zeros((T, 40))
    for g in range(G):
        exact[bounds[g]:bounds[g + 1]] = product(ex[bounds[g]:bounds[g + 1]], value[g])
    same(w4.grouped_matmul(x, q, gpu(bounds)), exact, kind)


@pytest.mark.parametrize("kind", SCALES)
def test_infinite_activations_in_a_captured_call(kind):
    r = rng(13)
    q, value, _ = coded(r, (136, 1024), 128, kind, True, -6, -5, whole=True)
    x, _ = dense(np.zeros((5, 1024)), kind)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w4.matmul(x, q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = w4.matmul(x, q)
    for k in range(4):
        ex = 64.0 * whole(r, (5, 1024))
        if k % 2:
            ex[k, 7] = np.inf
        x.copy_(torch.from_numpy(ex))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(y, product(ex, value), kind)
        same(w4.matmul(x, q), product(ex, value), kind)

"""A layer of experts in use: training steps captured and replayed, weights
shared by groups, and rows whose results do not depend on where they stand."""
import pytest

from dense_gemm_row_amd import grouped, w4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def whole(seed, shape, dtype, top=4):
    return torch.randint(-top, top + 1, shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def offsets_of(*bounds):
    return torch.tensor(bounds, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_captured_training_step(dtype):
    """Forward and backward pass in one graph, replayed with other rows and
    offsets, eager steps in between."""
    x, w, dy = whole(1, (200, 128), dtype), whole(2, (3, 128, 72), dtype), whole(3, (200, 72), dtype)
    at = offsets_of(0, 50, 50, 190)
    x.requires_grad_(True)
    w.requires_grad_(True)

    def step():
        y = grouped.linear(x, w, at)
        return (y.detach(), *torch.autograd.grad(y, (x, w), dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step()
    for k, bounds in enumerate([(0, 50, 50, 190), (10, 10, 100, 200), (0, 0, 0, 0), (0, 1, 2, 200)]):
        with torch.no_grad():
            x.copy_(whole(10 + k, x.shape, dtype))
            dy.copy_(whole(20 + k, dy.shape, dtype))
        at.copy_(offsets_of(*bounds))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        y, dx, dw = (torch.zeros_like(o, dtype=torch.float64) for o in outs)
        for g, (a, b) in enumerate(zip(bounds, bounds[1:])):
            xs, ws, ds = x.detach()[a:b].double(), w.detach()[g].double(), dy[a:b].double()
            y[a:b], dx[a:b], dw[g] = xs @ ws, ds @ ws.T.contiguous(), xs.T.contiguous() @ ds
        for got, exact in zip(outs, (y, dx, dw)):
            assert torch.equal(got, exact.to(dtype)), k


@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_a_capture_refuses_leaves_of_a_living_step_on_another_stream():
    """(Refused at the forward pass: nothing of the backward pass is captured.)"""
    x, w = whole(8, (40, 64), torch.float32), whole(9, (2, 64, 32), torch.float32).requires_grad_(True)
    at = offsets_of(0, 20, 40)
    alive = grouped.linear(x, w, at)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with pytest.raises(RuntimeError, match="earlier step on another stream"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            grouped.linear(x, w, at)
    with torch.cuda.stream(side):  # outside a capture streams may differ
        again = grouped.linear(x, w, at)
    torch.cuda.synchronize()
    assert torch.equal(alive, again)
    del alive, again
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = grouped.linear(x, w, at)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[:20], x[:20] @ w[0])


@pytest.mark.parametrize("transposed", [False, True])
def test_gradient_of_weights_that_all_groups_share(transposed):
    x, dy = whole(4, (90, 64), torch.float32), whole(5, (90, 48), torch.float32)
    w = whole(6, (48, 64) if transposed else (64, 48), torch.float32).requires_grad_(True)
    at = offsets_of(5, 30, 30, 80)
    grouped.linear(x, w.expand(3, *w.shape), at, transposed).backward(dy)
    exact = x[5:80].double().T.contiguous() @ dy[5:80].double()
    assert torch.equal(w.grad, (exact.T if transposed else exact).float())


@pytest.mark.parametrize("K", [1024, 1000])
def test_rows_do_not_depend_on_their_place(K):
    """The same rows of one expert at other places among the rows, behind other
    offsets: the same results bit for bit."""
    g = torch.Generator("cuda").manual_seed(7)
    q = w4.quantize(torch.randn(6, 264, K, generator=g, device="cuda", dtype=torch.bfloat16), group=64)
    w = torch.randn(6, K, 264, generator=g, device="cuda", dtype=torch.bfloat16)
    rows = torch.randn(20, K, generator=g, device="cuda", dtype=torch.bfloat16)
    first = {}
    for start, behind in ((0, 60), (3, 57), (37, 23), (60, 0)):
        x = torch.cat((torch.randn(start, K, generator=g, device="cuda", dtype=torch.bfloat16), rows,
                       torch.randn(behind, K, generator=g, device="cuda", dtype=torch.bfloat16)))
        at = offsets_of(0, 0, start // 2, start, start + 20, 80, 80)  # group 3 has them
        for name, y in (("w4", w4.grouped_matmul(x, q, at)), ("product", grouped.matmul(x, w, at))):
            assert torch.equal(first.setdefault(name, y[start:start + 20].clone()), y[start:start + 20]), (name, start)

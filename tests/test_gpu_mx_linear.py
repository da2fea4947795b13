"""mx.linear as a member of autograd's graph: what it saves, what it refuses,
and weights of either orientation."""
import pytest

from dense_gemm_row_amd import mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def layer(kind, t=70, k=96, n=40, seed=31):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, k, generator=g).to(TYPES[kind]).cuda().requires_grad_(True)
    w = (torch.randn(k, n, generator=g) / 8).to(TYPES[kind]).cuda().requires_grad_(True)
    dy = torch.randn(t, n, generator=g).to(TYPES[kind]).cuda()
    return x, w, dy


@pytest.mark.parametrize("kind", TYPES)
def test_checkpoint_is_a_saved_tensor(kind):
    """The 8-bit checkpoint passes through saved-tensor hooks, and what they
    hand back is what the backward pass reads."""
    x, w, dy = layer(kind)
    wq = mx.quantize(w.detach(), transposed=True)
    mx.linear(x, w, wq).backward(dy)
    want = w.grad.clone(), x.grad.clone()
    w.grad = x.grad = None
    packed = []

    def pack(t):
        packed.append(t)
        return t.cpu()

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.cuda()):
        y = mx.linear(x, w, wq)
    assert sorted(t.numel() for t in packed) == sorted([w.numel(), 96 * 96, 96 * 4])  # 3 blocks a feature
    y.backward(dy)
    assert torch.equal(w.grad, want[0]) and torch.equal(x.grad, want[1])


def test_frozen_weight_saves_no_checkpoint():
    x, w, dy = layer("bf16")
    packed = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (packed.append(t), t)[1], lambda t: t):
        y = mx.linear(x, w.detach(), mx.quantize(w.detach(), transposed=True))
    assert [t.shape for t in packed] == [w.shape]
    y.backward(dy)
    assert x.grad is not None and w.grad is None


def test_second_derivative_is_refused():
    """The kernels record no graph, so a derivative of the gradients would
    lack their terms."""
    x, w, _ = layer("f32")
    y = mx.linear(x, w, mx.quantize(w.detach(), transposed=True))
    dx, dw = torch.autograd.grad((y * y).sum(), (x, w), create_graph=True)
    for loss in ((dx * x).sum(), (dw * w).sum()):
        with pytest.raises(RuntimeError, match="once_differentiable"):
            loss.backward(retain_graph=True)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", [(70, 96, 40), (1, 33, 1), (5, 1, 7), (0, 64, 8)])
def test_weight_of_either_orientation(kind, shape):
    """w as the transpose of a row-major N x K parameter gives what its
    row-major copy gives."""
    x, w, dy = layer(kind, *shape)
    param = w.detach().t().contiguous().requires_grad_(True)
    wq = mx.quantize(param.detach())
    assert torch.equal(wq.codes, mx.quantize(w.detach(), transposed=True).codes)
    y = mx.linear(x, w, wq)
    y.backward(dy)
    x2 = x.detach().clone().requires_grad_(True)
    y2 = mx.linear(x2, param.t(), wq)
    y2.backward(dy)
    assert torch.equal(y, y2)
    assert torch.equal(param.grad.t(), w.grad)
    # dx: the same sums, maybe in another order: n additions in FP32 and the
    # result's rounding, on both sides.
    size = dy.double().abs() @ w.detach().double().abs().t()
    half = torch.finfo(TYPES[kind]).eps / 2
    n = shape[2]
    assert bool(((x.grad.double() - x2.grad.double()).abs() <= 2 * ((n + 8) * 2.0 ** -23 + half) * size).all())

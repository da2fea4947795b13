"""Refusals of mx.linear, at the forward call and before any launch.  CPU
only."""
import pytest

from dense_gemm_row_amd import mx

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("form", ["strided", "expanded", "one value"])
def test_weights_that_the_backward_pass_cannot_read(form):
    big = torch.zeros(64, 64)
    w = {"strided": big[::2, ::2], "expanded": big[:1, :32].expand(32, 32), "one value": big[:1, :1].expand(32, 32)}[form]
    with pytest.raises(ValueError, match="row-major"):
        mx.linear(torch.zeros(4, 32), w, mx.empty(32, 32, mx.E2M1, "cpu"))


def test_other_refusals():
    x, w, wq = torch.zeros(4, 32), torch.zeros(32, 64), mx.empty(64, 32, mx.E2M1, "cpu")
    with pytest.raises(TypeError):
        mx.linear(x.half(), w, wq)
    with pytest.raises(ValueError, match="coded form"):
        mx.linear(x, w.t(), wq)
    with pytest.raises(ValueError, match="devices"):
        mx.linear(x, w.to("meta"), wq)
    with pytest.raises(ValueError):  # (host tensors)
        mx.linear(x, w, wq)

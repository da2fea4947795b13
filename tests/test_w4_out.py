"""Stacks of results that share memory are refused: one expert's would be
written over another's.  CPU only."""
import pytest

from dense_gemm_row_amd import w4

torch = pytest.importorskip("torch")


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


@pytest.mark.parametrize("t", [u8(3, 6, 64), u8(3, 6, 80)[..., :64], u8(4, 8, 64)[:3, :6], u8(6, 3, 64).transpose(0, 1), u8(1, 6, 64),
                               u8(3, 1, 64), u8(1, 1, 64).expand(1, 1, 64), u8(0, 6, 64), u8(3, 0, 64), u8(1, 64).expand(3, 0, 64),
                               u8(3, 6, 1), u8(6, 3, 1).transpose(0, 1), u8(6, 64)[None]])
def test_results_apart(t):
    w4._apart(t, "out")


@pytest.mark.parametrize("t", [u8(6, 64).expand(3, 6, 64), u8(3, 1, 64).expand(3, 6, 64), u8(1, 1, 64).expand(3, 6, 64),
                               u8(1200).as_strided((3, 6, 64), (63, 200, 1)), u8(4000).as_strided((3, 6, 64), (320, 64, 1)),
                               u8(6, 1).expand(3, 6, 1)])
def test_results_that_overlap(t):
    with pytest.raises(ValueError, match="overlap"):
        w4._apart(t, "out")

"""The norm and its backward pass at sizes and rows that test_gpu_norm.py does not reach."""
import pytest
import torch

from test_gpu_norm import BF16, EPS, FP32, backward, check_backward, check_forward, fq, normal, rstd_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,C", [(5, 0), (0, 64), (0, 0)])
@pytest.mark.parametrize("row", [False, True])
def test_nothing(fq, T, C, row):
    x, w = torch.zeros(T, C, dtype=BF16, device="cuda"), torch.ones(C, device="cuda")
    for residual in (None, x.clone()):
        got = fq.fp8_rmsnorm(x, w, residual, scaling=fq.SCALE_ROW if row else fq.SCALE_TILE_1x128)
        assert got.y.shape == got.q.shape == got.h.shape == (T, C) and got.rstd.shape == (T,)

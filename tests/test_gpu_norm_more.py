"""The norm and its backward pass at sizes and rows that test_gpu_norm.py does not reach."""
import numpy as np
import pytest
import torch

from test_gpu_norm import (BF16, EPS, FP32, backward, check_backward, check_forward, f64, fq, inside, normal,  # noqa: F401
                           rstd_of)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,C", [(5, 0), (0, 64), (0, 0)])
@pytest.mark.parametrize("row", [False, True])
def test_nothing(fq, T, C, row):
    x, w = torch.zeros(T, C, dtype=BF16, device="cuda"), torch.ones(C, device="cuda")
    for residual in (None, x.clone()):
        got = fq.fp8_rmsnorm(x, w, residual, scaling=fq.SCALE_ROW if row else fq.SCALE_TILE_1x128)
        assert got.y.shape == got.q.shape == got.h.shape == (T, C) and got.rstd.shape == (T,)


# Blocks visit rows one after the other, the next one's loads under way: several
# rows a block for every number of threads a row has, and for rows too long to be
# held; rows moved in vectors and element by element.
MANY = [(9000, 200), (9001, 199), (3000, 1000), (3001, 1001), (2000, 2048), (2001, 2047), (1500, 4096), (1501, 4094),
        (1000, 8192), (1000, 8190), (700, 16384), (700, 16382), (500, 20000)]


def check_dweight(dy, h, rstd, dw):
    """A sum over T rows goes through at most T / 152 + 1 rows of a thread (a block on
    each of 152 SMs at least, where there are as many), 8 threads of a block, 15
    blocks' sums of a warp that joins them and 32 such warps: one rounding each, and two
    for a term."""
    n = f64(h) * f64(rstd)[:, None]
    want, size = (f64(dy) * n).sum(axis=0), np.abs(f64(dy) * n).sum(axis=0)
    inside(dw, want, size * (h.shape[0] / 152 + 1 + 8 + 15 + 32 + 2) * 2.0 ** -24, "dw")


@pytest.mark.parametrize("shape", MANY)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_forward_of_several_rows_a_block(fq, shape, dtype):
    C = shape[1]
    x, r = normal(shape, 60, 2.0, dtype), normal(shape, 61, 1.0, dtype)
    w = 1 + 0.3 * normal((C,), 62, 1.0, FP32)
    for row, residual in ((False, r), (True, None)):
        got = fq.fp8_rmsnorm(x.cuda(), w.cuda(), None if residual is None else residual.cuda(), EPS,
                             fq.SCALE_ROW if row else fq.SCALE_TILE_1x128)
        check_forward(fq, x, w, residual, EPS, row, got)
        if residual is not None:
            for at in (0, 1):
                both = [x.cuda(), r.cuda()]
                for a, b in zip(fq.fp8_rmsnorm(both[0], w.cuda(), both[1], EPS, h=both[at]), got):
                    assert torch.equal(a, b)


@pytest.mark.parametrize("shape", MANY)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_backward_of_several_rows_a_block(fq, shape, dtype):
    h, dy, dres = normal(shape, 63, 2.0, dtype), normal(shape, 64, 0.1, dtype), normal(shape, 65, 0.1, dtype)
    w, rstd = 1 + 0.3 * normal((shape[1],), 66, 1.0, FP32), rstd_of(h)
    for add in (dres, None):
        dx, dw = backward(fq, dy, h, w, rstd, add)
        check_backward(dy, h, w, rstd, add, dx, None)
        check_dweight(dy, h, rstd, dw)
    own = dy.cuda()
    again = fq.fp8_rmsnorm_backward(own, h.cuda(), w.cuda(), rstd.cuda(), dx=own)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_many_rows_with_everything(fq):
    """More elements than 32 bits count, with a residual, h, y and dresidual; rows
    between the ones that are checked are zeros, so dweight is those rows' sum."""
    T, C, some = 300_000, 8192, [0, 1, 151_999, 299_997, 299_998, 299_999]

    def spread(seed, scale=1.0):
        t = torch.zeros(T, C, dtype=BF16, device="cuda")
        few = normal((len(some), C), seed, scale)
        t[some] = few.cuda()
        return t, few

    (x, xs), (r, rs), w = spread(67), spread(68), normal((C,), 69)
    got = fq.fp8_rmsnorm(x, w.cuda(), r)
    part = fq.NormOutput(got.h[some], got.y[some], got.q[some], got.scales[:, some], got.rstd[some])
    check_forward(fq, xs, w, rs, EPS, False, part)
    h, rstd = got.h, got.rstd
    del got, x, r
    (dy, dys), (dres, dress) = spread(70, 0.1), spread(71, 0.1)
    dx, dw = fq.fp8_rmsnorm_backward(dy, h, w.cuda(), rstd, dresidual=dres)
    hs, rstds = h[some].cpu(), rstd[some].cpu()
    check_backward(dys, hs, w, rstds, dress, dx[some], None)
    check_dweight(dys, hs, rstds, dw)
    between = torch.ones(T, dtype=torch.bool, device="cuda")
    between[some] = False
    assert (dx.abs().amax(dim=1)[between] == 0).all()

"""RMS norm with an 8-bit output and its backward pass on the GPU against the
definitions in 64 bits, within bounds counted from fp32 roundings."""
import numpy as np
import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}   # half a step, relative
# rows held by a warp, by 256 and 512 threads, and too long to be held; ragged tiles
SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 130), (33, 256), (9, 1000), (17, 1024), (4, 2050), (6, 4096),
          (3, 6000), (2, 12296), (3, 16384), (2, 16391), (2, 20000), (700, 264)]
EPS = 1e-6


@pytest.fixture(scope="module")
def fq():
    import scaled_quantize_fp8_warp_gb300 as fq
    yield fq
    assert fq.device_status() == fq.OK


def normal(shape, seed, scale=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def inside(got, want, bound, what):
    """Within `bound` and the rounding of got's type (1e-40: fp32's smallest steps)."""
    err = np.abs(f64(got) - want)
    bad = ~(err <= bound + HALF[got.dtype] * (np.abs(want) + bound) + 1e-40)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3], np.nanmax(err))


def check_forward(fq, x, w, residual, eps, row, got, want_y=True):
    C = x.shape[1]
    h = x
    if residual is not None:
        h = (x.float() + residual.float()).to(x.dtype)
        assert torch.equal(got.h.cpu(), h)
    rstd, y = ref.norm(f64(h), f64(w), float(np.float32(eps)))
    e = ref.rstd_error(C)
    inside(got.rstd, rstd, rstd * e, "rstd")
    e = e + 2 * ref.U32
    if want_y:
        inside(got.y, y, np.abs(y) * e, "y")
    else:
        assert got.y is None
    s = ref.norm_scales(y, row)
    scales = got.scales.reshape(-1, x.shape[0]).t()
    inside(scales, s, s * e, "scales")
    # q stands for y / s, whose error is that of y, of s and of the quotient's
    # rounding; then half a step of E4M3
    v = y / np.repeat(f64(scales), C if row else 128, axis=1)[:, :C]
    off = np.abs(v) * (e + ref.U32)
    err = np.abs(ref.value(got.q.cpu().numpy(), ref.E4M3) - v)
    assert (err <= np.maximum(2.0 ** -4 * (np.abs(v) + off), 2.0 ** -10) + off).all(), err.max()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("row", [False, True])
def test_forward(fq, shape, dtype, row):
    T, C = shape
    x, r = normal(shape, 1, 2.0, dtype), normal(shape, 2, 1.0, dtype)
    w = 1 + 0.3 * normal((C,), 3, 1.0, FP32)
    for weight, residual, want_y in ((w, r, True), (w.to(BF16), None, False)):
        got = fq.fp8_rmsnorm(x.cuda(), weight.cuda(), None if residual is None else residual.cuda(), EPS,
                             fq.SCALE_ROW if row else fq.SCALE_TILE_1x128, want_y=want_y)
        check_forward(fq, x, weight, residual, EPS, row, got, want_y)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("C", [64, 512, 2048, 4096, 8192, 16384, 20480])
def test_bytes_are_the_casts(fq, dtype, C):
    """From an fp32 y the 8-bit output is, bit for bit, what the quantise calls
    give; from bf16 rows it is that of the y which a weight of bf16 rows in
    fp32 gives."""
    x, w = normal((48, C), 4, 1.5, dtype), 1 + 0.2 * normal((C,), 5, 1.0, FP32)
    y = fq.fp8_rmsnorm(x.float().cuda(), w.cuda(), eps=EPS, scaling=None).y
    q, s, _, _ = fq.fp8_quantize_tile1x128(y, fq.E4M3)
    got = fq.fp8_rmsnorm(x.cuda(), w.cuda(), eps=EPS, want_y=False)
    assert torch.equal(got.q, q) and torch.equal(got.scales, s)
    q, s, _, _ = fq.fp8_quantize_rowwise(y, fq.E4M3)
    got = fq.fp8_rmsnorm(x.cuda(), w.cuda(), eps=EPS, scaling=fq.SCALE_ROW)
    assert torch.equal(got.q, q) and torch.equal(got.scales, s)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("C", [40, 1024, 5000])
def test_rows_apart_and_unaligned(fq, dtype, C):
    """Slices of wider matrices, and rows that start on no 16-byte boundary."""
    wide = [normal((20, C + 24), k, 1.0, dtype).cuda() for k in range(6, 10)]
    w = (1 + 0.1 * normal((C + 1,), 10, 1.0, FP32)).cuda()[1:]   # 4-byte aligned
    for at in (0, 8, 3):
        x, r, h, y = (m[:, at:at + C] for m in wide)
        left = [m.clone() for m in wide[2:]]
        got = fq.fp8_rmsnorm(x, w, r, EPS, h=h, y=y)
        assert got.h is h and got.y is y
        check_forward(fq, x.cpu(), w.cpu(), r.cpu(), EPS, False, got)
        for m, was in zip(wide[2:], left):   # nothing beside the columns moved
            was[:, at:at + C] = m[:, at:at + C]
            assert torch.equal(m, was)


@pytest.mark.parametrize("C", [96, 3000, 17000])
def test_h_in_place(fq, C):
    x, r, w = normal((10, C), 11), normal((10, C), 12), normal((C,), 13)
    want = fq.fp8_rmsnorm(x.cuda(), w.cuda(), r.cuda(), EPS)
    for at in (0, 1):
        both = [x.cuda(), r.cuda()]
        got = fq.fp8_rmsnorm(both[0], w.cuda(), both[1], EPS, h=both[at])
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("row", [False, True])
def test_output_is_an_operand(fq, row):
    """The 8-bit output multiplied by a weight is what the cast of an fp32 y gives."""
    x, w = normal((200, 512), 50).cuda(), (1 + 0.2 * normal((512,), 51, 1.0, FP32)).cuda()
    weight = normal((256, 512), 52, 0.05).cuda()
    y = fq.fp8_rmsnorm(x.float(), w, eps=EPS, scaling=None).y
    G = fq.GemmOperand
    if row:
        q, s, _, _ = fq.fp8_quantize_rowwise(y, fq.E4M3)
        wq, ws, _, _ = fq.fp8_quantize_rowwise(weight, fq.E4M3)
        n = fq.fp8_rmsnorm(x, w, eps=EPS, scaling=fq.SCALE_ROW)
        a, b, c = G.row(q, fq.E4M3, s), G.row(n.q, fq.E4M3, n.scales), G.row(wq, fq.E4M3, ws)
    else:
        q, s, _, _ = fq.fp8_quantize_tile1x128(y, fq.E4M3)
        wq, _, ws = fq.fp8_quantize_block128x128(weight, fq.E4M3)
        n = fq.fp8_rmsnorm(x, w, eps=EPS)
        a, b, c = G.tile(q, fq.E4M3, s), G.tile(n.q, fq.E4M3, n.scales), G.block(wq, fq.E4M3, ws)
    assert torch.equal(fq.fp8_gemm_fprop(a, c), fq.fp8_gemm_fprop(b, c))


def test_another_stream_and_a_graph(fq):
    x, r, w = normal((90, 640), 53).cuda(), normal((90, 640), 54).cuda(), normal((640,), 55).cuda()

    def step(stream=None):
        n = fq.fp8_rmsnorm(x, w, r, EPS, stream=stream)
        return (*n, *fq.fp8_rmsnorm_backward(n.y, n.h, w, n.rstd, dresidual=x, stream=stream))
    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):   # two at once, each with storage of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    x.copy_(normal((90, 640), 56))
    for k, (g, _) in enumerate(graphs):
        with torch.cuda.stream(s if k else torch.cuda.current_stream()):
            if k:
                s.wait_stream(torch.cuda.default_stream())
            g.replay()
    torch.cuda.synchronize()
    want = step()
    for _, got in graphs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_zero_and_special_rows(fq):
    C = 300
    x = normal((7, C), 14, 1.0, FP32)
    x[0] = 0.0
    x[1, 5] = float("inf")
    x[2, 200] = float("nan")
    x[3] = -float("inf")
    x[4] = 1e25                    # squares past fp32: rstd is 0
    x[5] = 1e-30                   # squares below it: eps alone
    w = torch.ones(C)
    for row in (False, True):
        got = fq.fp8_rmsnorm(x.cuda(), w.cuda(), eps=EPS, scaling=fq.SCALE_ROW if row else fq.SCALE_TILE_1x128)
        y, q = got.y.cpu(), got.q.cpu()
        scales = got.scales.reshape(-1, 7).cpu()
        assert (y[0] == 0).all() and (q[0] & 0x7F == 0).all() and (scales[:, 0] == np.float32(1e-12)).all()
        assert y[1].isnan().sum() == 1 and y[1, 5].isnan() and got.rstd[1] == 0
        assert y[2].isnan().all() and y[3].isnan().all() and (q[2] & 0x7F == 0x7F).all()
        assert got.rstd[4] == 0 and (y[4] == 0).all()
        np.testing.assert_allclose(y[5].numpy(), 1e-27, rtol=1e-6)
        tiles = 1 if row else 3
        assert scales[0, 1].isnan()                       # the tile (row) that holds the NaN
        assert row or (scales[1:tiles, 1] == np.float32(1e-12)).all()
        check_forward(fq, x[6:], w, None, EPS, row, fq.fp8_rmsnorm(
            x[6:].cuda(), w.cuda(), eps=EPS, scaling=fq.SCALE_ROW if row else fq.SCALE_TILE_1x128))


def test_an_infinite_weight(fq):
    """y infinite without a NaN: the tile's scale is infinite, as the quantise call's."""
    x, w = normal((16, 256), 15, 1.0, FP32), torch.ones(256)
    w[130] = float("inf")
    got = fq.fp8_rmsnorm(x.cuda(), w.cuda(), eps=EPS)
    q, s, _, _ = fq.fp8_quantize_tile1x128(got.y, fq.E4M3)
    assert torch.equal(got.q, q) and torch.equal(got.scales, s) and got.scales[1].isinf().all()


def backward(fq, dy, h, w, rstd, dres, **more):
    c = lambda t: None if t is None else t.cuda()
    return fq.fp8_rmsnorm_backward(c(dy), c(h), c(w), c(rstd), dresidual=c(dres), **more)


def check_backward(dy, h, w, rstd, dres, dx, dw):
    want, want_w, err, err_w = ref.norm_backward(f64(dy), f64(h), f64(w), f64(rstd),
                                                 0.0 if dres is None else f64(dres))
    inside(dx, want, err, "dx")
    if dw is not None:
        assert dw.dtype == w.dtype
        inside(dw, want_w, err_w, "dw")


def rstd_of(h):
    return torch.from_numpy((1.0 / np.sqrt((f64(h) ** 2).mean(axis=1) + EPS)).astype(np.float32))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_backward(fq, shape, dtype):
    T, C = shape
    h, dy, dres = normal(shape, 20, 2.0, dtype), normal(shape, 21, 0.1, dtype), normal(shape, 22, 0.1, dtype)
    w, rstd = 1 + 0.3 * normal((C,), 23, 1.0, FP32), rstd_of(h)
    for weight, add in ((w, dres), (w.to(BF16), None)):
        check_backward(dy, h, weight, rstd, add, *backward(fq, dy, h, weight, rstd, add))
    dx, dw = backward(fq, dy, h, w, rstd, dres, want_dweight=False)
    assert dw is None
    check_backward(dy, h, w, rstd, dres, dx, None)


@pytest.mark.parametrize("C", [72, 1024, 4100, 16400])
def test_backward_rows_apart_and_in_place(fq, C):
    wide = [normal((30, C + 16), k, 0.5).cuda() for k in range(24, 27)]
    w = normal((C,), 27)
    for at in (0, 8, 5):
        h, dy, dres = (m[:, at:at + C] for m in wide)
        rstd = rstd_of(h)
        want = backward(fq, dy, h, w, rstd, dres)
        check_backward(dy, h, w, rstd, dres, *want)
        for which in (0, 1):
            own = [dy.clone(), dres.clone()]
            dx, dw = fq.fp8_rmsnorm_backward(own[0], h, w.cuda(), rstd.cuda(), dresidual=own[1], dx=own[which])
            assert dx is own[which] and torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_gradients_against_differences(fq):
    """dx and dw of L = sum dy y + sum dres h, by central differences of the
    definition in 64 bits; a step of 1e-4 leaves an error of its square."""
    T, C, step = 3, 20, 1e-4
    h, dy, dres = (normal((T, C), k, 1.0, FP32) for k in (30, 31, 32))
    w = 1 + 0.3 * normal((C,), 33, 1.0, FP32)
    loss = lambda h, w: (f64(dy) * ref.norm(h, w, EPS)[1]).sum() + (f64(dres) * h).sum()
    dx, dw = backward(fq, dy, h, w, rstd_of(h), dres)
    for t in range(T):
        for c in range(C):
            d = np.zeros((T, C))
            d[t, c] = step
            num = (loss(f64(h) + d, f64(w)) - loss(f64(h) - d, f64(w))) / (2 * step)
            assert abs(num - dx[t, c].item()) < 1e-5
    for c in range(C):
        d = np.zeros(C)
        d[c] = step
        num = (loss(f64(h), f64(w) + d) - loss(f64(h), f64(w) - d)) / (2 * step)
        assert abs(num - dw[c].item()) < 1e-5


def test_empty(fq):
    for T, C in ((0, 64), (5, 0)):
        x, w = torch.zeros(T, C, dtype=BF16).cuda(), torch.ones(C).cuda()
        got = fq.fp8_rmsnorm(x, w, x.clone())
        assert got.y.shape == (T, C)
        dx, dw = fq.fp8_rmsnorm_backward(x, x, w, torch.ones(T).cuda())
        assert dx.shape == (T, C) and (dw == 0).all()


def test_results_repeat(fq):
    x, w = normal((2000, 1504), 40).cuda(), normal((1504,), 41).cuda()
    rstd = fq.fp8_rmsnorm(x, w).rstd
    a, b = (fq.fp8_rmsnorm_backward(x, x, w, rstd) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_many_rows(fq):
    """More elements than 32 bits count, checked in its last rows."""
    T, C = 300_000, 8192
    x = torch.zeros(T, C, dtype=BF16, device="cuda")
    x[-3:] = normal((3, C), 42).cuda()
    x[0] = x[-1]
    w = normal((C,), 43)
    got = fq.fp8_rmsnorm(x, w.cuda(), want_y=False, scaling=fq.SCALE_ROW)
    for rows in (slice(T - 3, T), slice(0, 1)):
        part = fq.NormOutput(x[rows], None, got.q[rows], got.scales[rows], got.rstd[rows])
        check_forward(fq, x[rows].cpu(), w, None, EPS, True, part, want_y=False)
    rstd = got.rstd
    del got
    dx, dw = fq.fp8_rmsnorm_backward(x, x, w.cuda(), rstd)
    rows = slice(T - 3, T)
    check_backward(x[rows].cpu(), x[rows].cpu(), w, rstd[rows].cpu(), None, dx[rows], None)


def test_refusals(fq):
    x, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        fq.fp8_rmsnorm(x, w[:32])
    with pytest.raises(ValueError):
        fq.fp8_rmsnorm(x, w, x.float())
    with pytest.raises(ValueError):
        fq.fp8_rmsnorm(x, w, h=x)
    with pytest.raises(TypeError):
        fq.fp8_rmsnorm(x.half(), w)
    with pytest.raises(fq.Fp8qError):
        fq.fp8_rmsnorm(x, w, scaling=fq.SCALE_TENSOR)
    with pytest.raises(fq.Fp8qError):
        fq.fp8_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(ValueError):
        fq.fp8_rmsnorm_backward(x, x, w, torch.ones(3, device="cuda"))
    with pytest.raises(fq.Fp8qError):
        fq.fp8_rmsnorm_backward(x, x, w, torch.ones(4, device="cuda"),
                                workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))

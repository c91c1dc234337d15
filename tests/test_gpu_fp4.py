"""4-bit quantisation and products on the GPU against plain 64-bit definitions
(fp4_reference): codes and scale bytes bit for bit, products within the bound
of product_bound."""
import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu
KINDS = [0, 1]


@pytest.fixture(scope="module")
def fq():
    import scaled_quantize_fp8_warp_gb300 as fq
    yield fq
    assert fq.device_status() == fq.OK


def normal(shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f32(t):
    return t.detach().float().cpu().numpy()


def check_operand(op, x, kind, amax=None, what=""):
    """The operand is x [R, C] quantised, bit for bit, padding included."""
    codes, byte, g = ref.quantize(x, kind, amax)
    np.testing.assert_array_equal(op.data.cpu().numpy(), ref.pack(codes), err_msg=what + " codes")
    got = op.scales.cpu().numpy()
    want = ref.atoms(byte, kind, op.rows, op.K)
    np.testing.assert_array_equal(got, want, err_msg=what + " scales")
    if kind == 1:
        np.testing.assert_array_equal(op.global_scale.cpu().numpy()[0], g)


SHAPES = [(1, 1), (1, 16), (1, 4096), (3, 17), (31, 33), (32, 32), (128, 128), (129, 130),
          (257, 96), (100, 1000), (640, 48)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize(fq, kind, dtype, shape):
    x = normal(shape, 7, 0.3, dtype)
    x[::5] *= 300
    q, qt = fq.fp4_quantize(x.cuda(), kind, rows=True, cols=True)
    check_operand(q, f32(x), kind, what="rows")
    check_operand(qt, f32(x).T.copy(), kind, amax=np.abs(f32(x)).max(), what="cols")
    for op, v in ((q, f32(x)), (qt, f32(x).T.copy())):
        want = ref.dequantized(v, kind)
        got = fq.fp4_dequantize(op, out_dtype=torch.float32).cpu().numpy()
        np.testing.assert_array_equal(got, want.astype(np.float32))
        if kind == 0:   # few enough bits for bf16
            np.testing.assert_array_equal(f32(fq.fp4_dequantize(op)), want.astype(np.float32))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("want", [(True, False), (False, True)])
def test_quantize_one_orientation(fq, kind, want):
    x = normal((70, 200), 8)
    q, qt = fq.fp4_quantize(x.cuda(), kind, rows=want[0], cols=want[1])
    assert (q is not None, qt is not None) == want
    check_operand(q if want[0] else qt, f32(x) if want[0] else f32(x).T.copy(), kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("off,ld", [(0, 256), (1, 203), (8, 264), (3, 512)])
def test_quantize_slice_of_a_wider_matrix(fq, kind, dtype, off, ld):
    wide = normal((65, ld), 9, 2.0, dtype)
    x = wide[:, off:off + 200]
    q, qt = fq.fp4_quantize(wide.cuda()[:, off:off + 200], kind, rows=True, cols=True)
    check_operand(q, f32(x), kind)
    check_operand(qt, f32(x).T.copy(), kind, amax=np.abs(f32(x)).max())


@pytest.mark.parametrize("kind", KINDS)
def test_every_bf16_value(fq, kind):
    """All finite bf16 values, under block maxima that put them all over the
    codes and the ties between them."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    v = v[(v.abs() < 2.0 ** 100)].reshape(-1)
    x = torch.zeros((v.numel(), 32), dtype=torch.bfloat16)
    for j in range(32):   # each value beside its multiples by 1, 1.5, 1.25, ... up to 2^5
        x[:, j] = v * (1 + (j % 8) / 8) * 2.0 ** (j // 8)
    check = x[torch.isfinite(x).all(1)]
    amax = torch.full((1,), 6.0 * 448, dtype=torch.float32)
    q, _ = fq.fp4_quantize(check.cuda(), kind, amax=amax.cuda() if kind else None)
    check_operand(q, f32(check), kind, amax=6.0 * 448)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_what_is_not_finite(fq, kind, dtype):
    x = normal((40, 96), 10, 1.0, dtype)
    x[3, 5] = float("nan")
    x[7, 64] = float("inf")
    x[9, 95] = float("-inf")
    x[11] = 0.0
    x[12] = -0.0
    amax = torch.tensor([4.0])
    q, qt = fq.fp4_quantize(x.cuda(), kind, cols=True, amax=amax.cuda() if kind else None)
    check_operand(q, f32(x), kind, amax=4.0)
    check_operand(qt, f32(x).T.copy(), kind, amax=4.0)
    got = fq.fp4_dequantize(q, out_dtype=torch.float32).cpu()
    n = ref.BLOCK[kind]
    for r, c in ((3, 5), (7, 64), (9, 95)):
        assert torch.isnan(got[r, c // n * n:(c // n + 1) * n]).all()
        got[r, c // n * n:(c // n + 1) * n] = 0
    assert torch.isfinite(got).all()


def test_nvfp4_amax_that_is_not_finite_is_nan_everywhere(fq):
    x = normal((20, 64), 11)
    x[2, 3] = float("inf")
    q, _ = fq.fp4_quantize(x.cuda(), fq.NVFP4)
    assert torch.isnan(fq.fp4_dequantize(q)).all()
    w, _ = fq.fp4_quantize(normal((32, 64), 12).cuda(), fq.NVFP4)
    assert torch.isnan(fq.fp4_gemm(q, w)).all()
    assert torch.isnan(fq.fp4_linear(x.cuda(), w)).all()
    x[2, 3] = float("nan")
    assert torch.isnan(fq.fp4_linear(x.cuda(), w)).all()


@pytest.mark.parametrize("amax", [0.0, 1e-30, 0.01, 1e30])
def test_nvfp4_calibrated_amax(fq, amax):
    """An amax far from the tensor's: elements saturate or vanish, all finite."""
    x = normal((33, 160), 13, 1.0, torch.float32)
    x[4] *= 1e30
    t = torch.tensor([amax], dtype=torch.float32)
    q, qt = fq.fp4_quantize(x.cuda(), fq.NVFP4, cols=True, amax=t.cuda())
    check_operand(q, f32(x), 1, amax=amax)
    check_operand(qt, f32(x).T.copy(), 1, amax=amax)


@pytest.mark.parametrize("kind", KINDS)
def test_zero_sizes(fq, kind):
    for shape in ((0, 64), (5, 0)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        q, qt = fq.fp4_quantize(x, kind, cols=True)
        assert fq.fp4_dequantize(q).shape == shape
    w, _ = fq.fp4_quantize(normal((32, 64), 1).cuda(), kind)
    assert fq.fp4_linear(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w).shape == (0, 32)
    e, _ = fq.fp4_quantize(torch.empty((5, 0), dtype=torch.bfloat16, device="cuda"), kind)
    f, _ = fq.fp4_quantize(torch.empty((7, 0), dtype=torch.bfloat16, device="cuda"), kind)
    assert (fq.fp4_gemm(e, f) == 0).all()
    y, dx, dw = fq.fp4_linear_train(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"),
                                    normal((32, 64), 1).cuda(),
                                    torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"), kind)
    assert y.shape == (0, 32) and (dw == 0).all() and dw.shape == (32, 64)


PRODUCTS = [(1, 1, 1), (1, 16, 32), (1, 4096, 4096), (2, 300, 1000), (8, 128, 256), (9, 131, 259),
            (16, 1000, 8192), (17, 264, 520), (33, 96, 64), (64, 512, 1024), (65, 129, 96),
            (128, 256, 256), (129, 257, 513), (250, 640, 192), (300, 1000, 2010), (640, 1536, 640),
            (257, 16, 4096), (40, 50, 16384)]


def check_product(got, a, b, bf16):
    want = a @ b.T
    err = np.abs(f32(got).astype(np.float64) - want)
    bound = ref.product_bound(a, b, bf16)
    bad = err > bound
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3], (err / np.maximum(bound, 1e-300)).max())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", PRODUCTS)
def test_gemm_and_linear(fq, kind, out, size):
    M, N, K = size
    x, w = normal((M, K), M + 1), normal((N, K), N + 2, 0.02)
    qx, _ = fq.fp4_quantize(x.cuda(), kind)
    qw, _ = fq.fp4_quantize(w.cuda(), kind)
    a, b = ref.dequantized(f32(x), kind), ref.dequantized(f32(w), kind)
    check_product(fq.fp4_gemm(qx, qw, out_dtype=out), a, b, out == torch.bfloat16)
    check_product(fq.fp4_linear(x.cuda(), qw, out_dtype=out), a, b, out == torch.bfloat16)
    if kind == fq.NVFP4:
        amax = torch.tensor([2.5], device="cuda")
        check_product(fq.fp4_linear(x.cuda(), qw, x_amax=amax, out_dtype=out),
                      ref.dequantized(f32(x), kind, 2.5), b, out == torch.bfloat16)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 5, 16, 40, 200])
def test_linear_reads_fp32_and_strided_rows(fq, kind, M):
    K, N = 1000, 520
    for dtype, off, ld in ((torch.float32, 0, K), (torch.float32, 3, K + 5), (torch.bfloat16, 8, K + 24),
                           (torch.bfloat16, 1, K + 7)):
        wide = normal((M, ld), 21, 1.0, dtype)
        w = normal((N, K), 22, 0.02)
        qw, _ = fq.fp4_quantize(w.cuda(), kind)
        got = fq.fp4_linear(wide.cuda()[:, off:off + K], qw, out_dtype=torch.float32)
        check_product(got, ref.dequantized(f32(wide[:, off:off + K]), kind),
                      ref.dequantized(f32(w), kind), False)


@pytest.mark.parametrize("kind", KINDS)
def test_a_row_with_a_nan_leaves_the_others(fq, kind):
    for M in (3, 40, 300):
        x, w = normal((M, 320), 31), normal((48, 320), 32)
        x[1, 100] = float("nan")
        amax = torch.tensor([4.0], device="cuda")
        qw, _ = fq.fp4_quantize(w.cuda(), kind)
        y = fq.fp4_linear(x.cuda(), qw, x_amax=amax if kind else None, out_dtype=torch.float32)
        assert torch.isnan(y[1]).all()
        keep = [i for i in range(M) if i != 1]
        check_product(y[keep], ref.dequantized(f32(x[keep]), kind, 4.0),
                      ref.dequantized(f32(w), kind), False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [(1, 16, 33), (96, 64, 160), (200, 130, 257), (512, 384, 256)])
def test_linear_train(fq, kind, out, size):
    M, N, K = size
    x, w, g = normal((M, K), 41), normal((N, K), 42, 0.02), normal((M, N), 43, 1e-3)
    y, dx, dw = fq.fp4_linear_train(x.cuda(), w.cuda(), g.cuda(), kind, out_dtype=out)
    q = lambda t: ref.dequantized(f32(t), kind)
    q_t = lambda t: ref.dequantized(f32(t).T.copy(), kind)
    bf = out == torch.bfloat16
    check_product(y, q(x), q(w), bf)
    check_product(dx, q(g), q_t(w), bf)
    check_product(dw, q_t(g), q_t(x), bf)


def test_linear_train_is_the_gradient_of_the_product(fq):
    """Where 4 bits hold every value exactly, dx and dw are the derivatives of
    sum(g * x w^T): differences of the forward product along single elements."""
    pick = lambda shape, seed: torch.from_numpy(np.random.default_rng(seed).choice(
        [-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 2.0], shape)).to(torch.bfloat16)
    M, N, K = 64, 96, 160
    x, w, g = pick((M, K), 1), pick((N, K), 2), pick((M, N), 3)
    for t in (x, w, g):      # every block's maximum is 4: its scale is 1, and 0.5 .. 4 are codes
        t[::8, ::8] = 4.0
    _, dx, dw = fq.fp4_linear_train(x.cuda(), w.cuda(), g.cuda(), fq.MXFP4, out_dtype=torch.float32)
    loss = lambda x, w: float((g.double() * (x.double() @ w.double().T)).sum())
    for i, j in ((0, 0), (5, 9), (63, 159)):
        up, down = x.clone(), x.clone()
        up[i, j] += 0.5
        down[i, j] -= 0.5
        assert float(dx[i, j]) == loss(up, w) - loss(down, w)
    for i, j in ((0, 1), (50, 70), (95, 159)):
        up, down = w.clone(), w.clone()
        up[i, j] += 0.5
        down[i, j] -= 0.5
        assert float(dw[i, j]) == loss(x, up) - loss(x, down)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 24, 400])
def test_same_bits_again_and_on_another_stream(fq, kind, M):
    x, w = normal((M, 2048), 51).cuda(), normal((768, 2048), 52).cuda()
    qw, _ = fq.fp4_quantize(w, kind)
    first = fq.fp4_linear(x, qw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [fq.fp4_linear(x, qw, stream=s) for _ in range(5)]
    torch.cuda.current_stream().wait_stream(s)
    for y in got:
        assert torch.equal(first, y)


@pytest.mark.parametrize("M", [2, 300])
def test_linear_in_a_graph(fq, M):
    x, w = normal((M, 512), 61).cuda(), normal((256, 512), 62).cuda()
    qw, _ = fq.fp4_quantize(w, fq.NVFP4)
    ws = torch.empty(fq.fp4_linear_workspace_size(fq.NVFP4, M, 256, 512), dtype=torch.uint8,
                     device="cuda")
    y = torch.empty((M, 256), dtype=torch.bfloat16, device="cuda")
    fq.fp4_linear(x, qw, workspace=ws, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.fp4_linear(x, qw, workspace=ws, out=y)
    new = normal((M, 512), 63, 3.0)
    x.copy_(new.cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, fq.fp4_linear(new.cuda(), qw))


def test_offsets_past_32_bits(fq):
    """Rows whose byte offsets pass 2^32 (x, codes) and outputs past 2^31
    elements come out as the same rows do alone."""
    R, C = 140000, 32768
    x = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    x[-300:] = normal((300, C), 71).cuda()
    q, qt = fq.fp4_quantize(x, fq.MXFP4, cols=True)
    alone, _ = fq.fp4_quantize(x[-300:].contiguous(), fq.MXFP4)
    assert torch.equal(q.data[-300:], alone.data)
    v = fq.fp4_dequantize(q)
    assert torch.equal(v[-300:], fq.fp4_dequantize(alone))
    assert not v[:-300].any()
    v = fq.fp4_dequantize(qt)
    assert torch.equal(v[-1, -32 * (300 // 32):],
                       fq.fp4_dequantize(fq.fp4_quantize(x[-32 * (300 // 32):, -1:].contiguous(),
                                                         fq.MXFP4, rows=False, cols=True)[1])[0])
    del x, q, qt, v
    M, N = 66000, 33000
    a, b = normal((M, 64), 72).cuda(), normal((N, 64), 73).cuda()
    qa, qb = fq.fp4_quantize(a, fq.MXFP4)[0], fq.fp4_quantize(b, fq.MXFP4)[0]
    y = fq.fp4_gemm(qa, qb)
    tail = fq.fp4_gemm(fq.fp4_quantize(a[-130:].contiguous(), fq.MXFP4)[0], qb)
    assert torch.equal(y[-130:], tail)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [(1, 12288, 4096), (2, 4096, 16384), (13, 4096, 16384),
                                  (16, 16384, 4096), (48, 12288, 4096), (128, 4096, 16384),
                                  (500, 1000, 16384), (300, 4096, 8192)])
def test_few_rows_of_a_layer(fq, kind, size):
    """Rings that wrap and clusters of every size, against a 64-bit product of
    the values the operands stand for."""
    M, N, K = size
    x, w = normal((M, K), 81).cuda(), normal((N, K), 82, 0.02).cuda()
    qx, qw = fq.fp4_quantize(x, kind)[0], fq.fp4_quantize(w, kind)[0]
    a = fq.fp4_dequantize(qx, out_dtype=torch.float32).double()
    b = fq.fp4_dequantize(qw, out_dtype=torch.float32).double()
    want, mag = a @ b.T, a.abs() @ b.abs().T
    bound = (K / 64 + 12) * 2.0 ** -23 * mag + 2.0 ** -23 * want.abs()
    for y in (fq.fp4_linear(x, qw, out_dtype=torch.float32),
              fq.fp4_gemm(qx, qw, out_dtype=torch.float32)):
        assert ((y.double() - want).abs() <= bound).all()

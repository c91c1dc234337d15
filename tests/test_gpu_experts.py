"""MXFP8 operands in groups and the experts' products on the GPU: casts bit for
bit against the definitions, products against 64 bits within bounds counted
from fp32 roundings, everything that no group owns left alone."""
import numpy as np
import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}   # half a step, relative
MARK = 0xAB

# rows of every group, and rows behind them
SPLITS = [([1], 0), ([0, 0, 0], 5), ([5], 300), ([0, 1, 0, 2], 3), ([127, 128, 129], 0), ([256, 1, 257, 0, 300], 17),
          ([130] * 9, 1), ([700], 0), ([0] * 40 + [3] + [0] * 23, 0)]


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


def ends_of(sizes):
    return [0] + np.cumsum(sizes).tolist()


def offsets_of(ends):
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


def marked(fq, rows, cols, groups, fmt, offsets, by_rows=True, transposed=True):
    op = fq.ExpertsOperand.empty(rows, cols, groups, "cuda", fmt, offsets, by_rows, transposed)
    for t in (op.q, op.q_scales, op.q_t, op.qt_scales):
        if t is not None:
            t.fill_(MARK)
    return op


def arrays(op):
    return {k: getattr(op, k).cpu().numpy() for k in ("q", "q_scales", "q_t", "qt_scales")
            if getattr(op, k) is not None}


def check_cast(fq, x, op, groups, index=None, rows=True, cols=True):
    """x on the host; op as the call left it, marked before."""
    xs = f64(x)
    if index is not None:
        picked = np.zeros((len(index), x.shape[1]))
        ok = (index >= 0) & (index < x.shape[0])
        picked[ok] = xs[index[ok]]
        xs = picked
    got = arrays(op)
    want = {k: np.full_like(v, MARK) for k, v in got.items()}
    ref.cast(xs, groups, op.fmt, want, rows, cols)
    for k in got:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)


def operand(fq, x, sizes, spare, fmt, **how):
    """The operand of x [sum(sizes), C] with `spare` rows behind, and its groups."""
    ends = ends_of(sizes)
    off = offsets_of(ends)
    op = marked(fq, ends[-1] + spare, x.shape[1], len(sizes), fmt, off, **how)
    x = torch.cat((x, torch.full((spare, x.shape[1]), float("nan"), dtype=x.dtype)))
    fq.fp8_quantize_experts(x.cuda(), len(sizes), off, rows=op.q is not None, cols=op.q_t is not None, fmt=fmt, out=op)
    return op, ref.Groups(ends)


def weights(fq, w, E, fmt=0, **how):
    """The operand of E weights [N, K] below one another."""
    op = marked(fq, w.shape[0], w.shape[1], E, fmt, None, **how)
    fq.fp8_quantize_experts(w.cuda(), E, rows=op.q is not None, cols=op.q_t is not None, fmt=fmt, out=op)
    return op, ref.Groups([w.shape[0] // E * e for e in range(E + 1)], equal=True)


# ------------------------------------------------------------------- the cast

@pytest.mark.parametrize("sizes,spare", SPLITS)
@pytest.mark.parametrize("C", [16, 144, 400])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("fmt", [0, 1])
def test_cast(fq, sizes, spare, C, dtype, fmt):
    x = normal((sum(sizes), C), 1, 1.0, dtype)
    if x.shape[0] > 2:
        x[1] *= 300.0
        x[2] *= 1e-3
    op, groups = operand(fq, x, sizes, spare, fmt)
    check_cast(fq, x, op, groups)


@pytest.mark.parametrize("E,n", [(1, 128), (3, 16), (4, 200), (5, 384), (7, 1)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_cast_equal_groups(fq, E, n, fmt):
    w = normal((E * n, 272), 2, 0.02)
    op, groups = weights(fq, w, E, fmt)
    check_cast(fq, w, op, groups)


def test_cast_is_the_dense_one(fq):
    """One group: fp8_quantize_mxfp8's bytes and scales."""
    x = normal((256, 384), 3).cuda()
    q, s, q_t, s_t = fq.fp8_quantize_mxfp8(x, fq.E4M3, cols=True)
    for off in (None, offsets_of([0, 256])):
        op = fq.fp8_quantize_experts(x, 1, off, cols=True)
        assert torch.equal(op.q, q) and torch.equal(op.q_scales[:s.numel()], s.view(-1))
        assert torch.equal(op.q_t[:, :256], q_t)
        if off is None:
            assert torch.equal(op.qt_scales, s_t.view(-1))


@pytest.mark.parametrize("rows,cols", [(True, False), (False, True), (True, True)])
def test_cast_gathers(fq, rows, cols):
    """Tokens that go to several experts, and indexes that are no token's."""
    T, C, sizes, spare = 70, 208, [40, 0, 150, 3], 9
    x = normal((T, C), 4)
    ends = ends_of(sizes)
    g = torch.Generator().manual_seed(5)
    index = torch.randint(0, T, (ends[-1] + spare,), generator=g, dtype=torch.int32)
    index[3], index[50], index[60] = -1, T, 2 ** 31 - 1
    off = offsets_of(ends)
    op = marked(fq, ends[-1] + spare, C, len(sizes), 0, off)
    fq.fp8_quantize_experts(x.cuda(), len(sizes), off, index.cuda(), rows=rows, cols=cols, out=op)
    check_cast(fq, x, op, ref.Groups(ends), index.numpy(), rows, cols)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("at", [0, 8, 1])
def test_cast_rows_apart(fq, dtype, at):
    wide = normal((150, 170), 6, 1.0, dtype)
    x = wide[:, at:at + 160]
    off = offsets_of([0, 20, 150])
    op = marked(fq, 150, 160, 2, 0, off)
    fq.fp8_quantize_experts(wide.cuda()[:, at:at + 160], 2, off, cols=True, out=op)
    check_cast(fq, x, op, ref.Groups([0, 20, 150]))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_cast_special_values(fq, dtype):
    x = normal((160, 96), 7, 1.0, dtype)
    x[0, 3], x[40, 50], x[70, 64] = float("nan"), float("inf"), -float("inf")
    x[80, :32] = 0.0
    x[81, :32] = -0.0
    x[82] = 1e-38
    x[83, 5] = torch.finfo(dtype).max
    x[84] = torch.finfo(dtype).tiny
    x[85] = 447.0
    x[86, :4] = torch.tensor([511.0, -511.0, 2 ** -10, -(2.0 ** -20)])
    for fmt in (0, 1):
        op, groups = operand(fq, x, [30, 130], 4, fmt)
        check_cast(fq, x, op, groups)


@pytest.mark.parametrize("bad", [[0, 50, 20, 70], [-5, 10, 90, 4000], [0, 70, 70, 2 ** 31 - 1], [60, 10, 0, 0],
                                 [-(2 ** 31), -1, 0, 12]])
def test_offsets_that_are_none_stay_inside(fq, bad):
    """Whatever the offsets hold, nothing outside the operand or the result is written."""
    S, C, N, E = 70, 64, 48, 3
    off = offsets_of(bad)
    guard = torch.full((3, S, C), MARK, dtype=torch.uint8, device="cuda")
    op = fq.ExpertsOperand.empty(S, C, E, "cuda", 0, off, True, True)
    op.struct.q = guard[1].data_ptr()
    fq.fp8_quantize_experts(normal((S, C), 8).cuda(), E, off, cols=True, out=op)
    w, _ = weights(fq, normal((E * N, C), 9), E)
    out = torch.full((3, S, N), 7.0, dtype=FP32, device="cuda")
    fq.fp8_experts_fprop(op, w, out=out[1])
    g = fq.fp8_quantize_experts(normal((S, N), 10).cuda(), E, off, cols=True)
    dw = torch.full((3, E, N, C), 7.0, dtype=FP32, device="cuda")
    fq.fp8_experts_wgrad(g, op, out=dw[1])
    torch.cuda.synchronize()
    for t, mark in ((guard, MARK), (out, 7.0), (dw, 7.0)):
        assert (t[0] == mark).all() and (t[2] == mark).all()


# --------------------------------------------------------------- the products

def bound(K, ab):
    """The tensor cores add K / 32 partial sums in fp32, truncating: one last
    place each, and a few within and behind them."""
    return (K / 32 + 12) * 2.0 ** -23 * ab


def near(got, a, b, what):
    """got = a . b^T of values in 64 bits."""
    want, err = a @ b.T, np.abs(f64(got) - a @ b.T)
    lim = bound(a.shape[1], np.abs(a) @ np.abs(b).T)
    lim = lim + HALF[got.dtype] * (np.abs(want) + lim) + 1e-40
    bad = ~(err <= lim)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3], err.max())


def check_rows_product(fq, sizes, spare, N, K, out, dgrad, fmt=0):
    S = sum(sizes)
    x, w = normal((S, N if dgrad else K), 11), normal((len(sizes) * N, K), 12, 0.05)
    op, groups = operand(fq, x, sizes, spare, fmt, transposed=False)
    wop, wgroups = weights(fq, w, len(sizes), by_rows=not dgrad, transposed=dgrad)
    result = torch.full((S + spare, K if dgrad else N), 3.0, dtype=out, device="cuda")
    op.q[S:] = 0x7F   # NaN where nobody's rows are
    f = fq.fp8_experts_dgrad if dgrad else fq.fp8_experts_fprop
    assert f(op, wop, out=result) is result
    assert (result[S:] == 3.0).all()
    rows = ref.group_rows(arrays(op), groups, fmt)
    ws = (ref.group_cols if dgrad else ref.group_rows)(arrays(wop), wgroups, 0)
    for (e, a, z, _), xv, wv in zip(groups, rows, ws):
        if z > a:
            near(result[a:z], xv, wv, (e, a, z))


@pytest.mark.parametrize("sizes,spare", SPLITS)
@pytest.mark.parametrize("N,K", [(16, 16), (144, 80), (272, 400), (528, 128)])
@pytest.mark.parametrize("dgrad", [False, True])
def test_rows_products(fq, sizes, spare, N, K, dgrad):
    check_rows_product(fq, sizes, spare, N, K, FP32 if (N + K) % 32 else BF16, dgrad)


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dgrad", [False, True])
def test_formats_and_types(fq, out, fmt, dgrad):
    check_rows_product(fq, [33, 0, 290, 5], 8, 400, 336, out, dgrad, fmt)


@pytest.mark.parametrize("K", [4096, 8208])
def test_long_contractions_and_many_tiles(fq, K):
    check_rows_product(fq, [3, 600, 0, 257, 31], 0, 1040, K, BF16, False)


@pytest.mark.parametrize("sizes,spare", [([1], 0), ([0, 2, 0, 1], 0), ([100], 27), ([17, 0, 31], 60), ([1] * 9, 1),
                                         ([127], 0), ([0, 0], 9)])
@pytest.mark.parametrize("N,K", [(144, 2048), (272, 4112), (1040, 4096)])
@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("dgrad", [False, True])
def test_few_rows(fq, sizes, spare, N, K, out, dgrad):
    """Fewer than 128 rows, whose contraction (4096 or so) is split over a cluster."""
    if dgrad:
        N, K = 16 * (K // 16), N
    check_rows_product(fq, sizes, spare, N, K, out, dgrad)


def test_many_experts(fq):
    g = np.random.default_rng(13)
    check_rows_product(fq, g.integers(0, 6, 1024).tolist(), 10, 48, 64, BF16, False)


@pytest.mark.parametrize("sizes,spare", SPLITS)
@pytest.mark.parametrize("N,K,out", [(16, 16, FP32), (144, 272, BF16), (400, 304, FP32), (272, 528, BF16)])
def test_wgrad(fq, sizes, spare, N, K, out):
    g, x = normal((sum(sizes), N), 14, 0.1), normal((sum(sizes), K), 15)
    gop, groups = operand(fq, g, sizes, spare, 1, by_rows=False)
    xop, _ = operand(fq, x, sizes, spare, 0, by_rows=False)
    dw = torch.full((len(sizes), N, K), 5.0, dtype=out, device="cuda")
    fq.fp8_experts_wgrad(gop, xop, out=dw)
    for (e, a, z, _), gv, xv in zip(groups, ref.group_cols(arrays(gop), groups, 1),
                                    ref.group_cols(arrays(xop), groups, 0)):
        if z > a:
            near(dw[e], gv, xv, e)
        else:
            assert (dw[e] == 0).all()


EMPTY = ["1010011010", "0101", "1000001000001", "111000", "1" + "0" * 30 + "11", "01" * 16, "0011" * 8, "100" * 11]


@pytest.mark.parametrize("present", EMPTY)
@pytest.mark.parametrize("out", [BF16, FP32])
def test_wgrad_with_empty_groups_between(fq, present, out):
    """As many tiles a group as CTA pairs run at once: every pair meets every
    group, those with no rows in any order with the others, time after time."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    N, K = 16, (128 if out == FP32 else 256) * pairs
    sizes = [int(c) * (1 + 37 * i % 150) for i, c in enumerate(present)]
    g, x = normal((sum(sizes), N), 40, 0.1), normal((sum(sizes), K), 41)
    gop, groups = operand(fq, g, sizes, 3, 1, by_rows=False)
    xop, _ = operand(fq, x, sizes, 3, 0, by_rows=False)
    dw = torch.full((len(sizes), N, K), 5.0, dtype=out, device="cuda")
    first = fq.fp8_experts_wgrad(gop, xop, out=dw).clone()
    torch.cuda.synchronize()
    assert fq.device_status() == fq.OK
    for (e, a, z, _), gv, xv in zip(groups, ref.group_cols(arrays(gop), groups, 1),
                                    ref.group_cols(arrays(xop), groups, 0)):
        if z > a:
            near(first[e], gv, xv, e)
        else:
            assert (first[e] == 0).all()
    for _ in range(20):
        dw.fill_(5.0)
        assert torch.equal(fq.fp8_experts_wgrad(gop, xop, out=dw), first)


@pytest.mark.parametrize("E,N,K,seed", [(1024, 16, 48, 42), (128, 112, 1600, 43), (83, 272, 528, 44),
                                        (31, 1040, 272, 45)])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_wgrad_of_many_groups_many_empty(fq, E, N, K, seed, out):
    r = np.random.default_rng(seed)
    sizes = (r.integers(0, 2, E) * r.integers(1, 40, E)).tolist()
    g, x = normal((sum(sizes), N), seed, 0.1), normal((sum(sizes), K), seed + 100)
    gop, groups = operand(fq, g, sizes, 0, 1, by_rows=False)
    xop, _ = operand(fq, x, sizes, 0, 0, by_rows=False)
    dw = fq.fp8_experts_wgrad(gop, xop, out=torch.full((E, N, K), 5.0, dtype=out, device="cuda"))
    torch.cuda.synchronize()
    assert fq.device_status() == fq.OK
    for (e, a, z, _), gv, xv in zip(groups, ref.group_cols(arrays(gop), groups, 1),
                                    ref.group_cols(arrays(xop), groups, 0)):
        if z > a:
            near(dw[e], gv, xv, e)
        else:
            assert (dw[e] == 0).all()


@pytest.mark.parametrize("out", [BF16, FP32])
@pytest.mark.parametrize("sizes", [[130, 0, 300, 5, 0, 60], [20] * 6])
def test_rows_products_of_many_tiles(fq, sizes, out):
    """Five tiles and more for every CTA pair, tiles of 128 and 256 rows."""
    check_rows_product(fq, sizes, 2, 16384, 48, out, False)


def test_equal_groups_of_tokens(fq):
    """x in equal groups, as experts of fixed capacity have: the same as offsets that say so."""
    x, w, g = normal((3 * 70, 96), 16), normal((3 * 64, 96), 17), normal((3 * 70, 64), 18)
    wop, _ = weights(fq, w, 3)
    off = offsets_of([0, 70, 140, 210])
    a = [fq.fp8_quantize_experts(t.cuda(), 3, cols=True) for t in (x, g)]
    b = [fq.fp8_quantize_experts(t.cuda(), 3, off, cols=True) for t in (x, g)]
    assert torch.equal(fq.fp8_experts_fprop(a[0], wop), fq.fp8_experts_fprop(b[0], wop))
    assert torch.equal(fq.fp8_experts_dgrad(a[1], wop), fq.fp8_experts_dgrad(b[1], wop))
    assert torch.equal(fq.fp8_experts_wgrad(a[1], a[0]), fq.fp8_experts_wgrad(b[1], b[0]))


def test_gradients_are_differences(fq):
    """Whole numbers up to 8 are exact in MXFP8 and their sums in fp32, so the
    products are too: L = sum g y is linear in x and in w, and its differences
    along any direction are what the gradients give, to the last bit."""
    sizes, N, K = [20, 0, 45], 48, 80
    r = np.random.default_rng(19)
    whole = lambda *s: torch.from_numpy(r.integers(-8, 9, s).astype(np.float32))
    x, w, g = whole(65, K), whole(3 * N, K), whole(65, N)
    off = offsets_of(ends_of(sizes))
    cast = lambda t: fq.fp8_quantize_experts(t.cuda(), 3, off, cols=True)
    fprop = lambda x, w: f64(fq.fp8_experts_fprop(cast(x), fq.fp8_quantize_experts(w.cuda(), 3), out_dtype=FP32))
    dx = f64(fq.fp8_experts_dgrad(cast(g), fq.fp8_quantize_experts(w.cuda(), 3, cols=True), out_dtype=FP32))
    dw = f64(fq.fp8_experts_wgrad(cast(g), cast(x), out_dtype=FP32)).reshape(3 * N, K)
    y = fprop(x, w)
    for k in range(4):
        to = whole(65, K)
        assert (f64(g) * (fprop(to, w) - y)).sum() == (dx * (f64(to) - f64(x))).sum()
        to = whole(3 * N, K)
        assert (f64(g) * (fprop(x, to) - y)).sum() == (dw * (f64(to) - f64(w))).sum()


# ------------------------------------------------------ streams, graphs, sizes

def test_another_stream(fq):
    x, w = normal((300, 256), 20).cuda(), normal((2 * 128, 256), 21).cuda()
    off = offsets_of([0, 100, 300])
    want = fq.fp8_experts_fprop(fq.fp8_quantize_experts(x, 2, off), fq.fp8_quantize_experts(w, 2))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    xs = fq.fp8_quantize_experts(x, 2, off, stream=s)
    got = fq.fp8_experts_fprop(xs, fq.fp8_quantize_experts(w, 2, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_graph_replays_with_other_groups(fq):
    """Captured once; rows, index and offsets change between replays on the device."""
    T, C, N, E, S = 64, 160, 96, 4, 200
    x, index = torch.zeros(T, C, dtype=BF16, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    w = fq.fp8_quantize_experts(normal((E * N, C), 22).cuda(), E, cols=True)
    op, y = marked(fq, S, C, E, 0, off), torch.zeros(S, N, device="cuda")
    dw = torch.zeros(E, N, C, device="cuda")
    gy = normal((S, N), 23).cuda()

    def step():
        fq.fp8_quantize_experts(x, E, off, index, cols=True, out=op)
        fq.fp8_experts_fprop(op, w, out=y)
        fq.fp8_experts_wgrad(fq.fp8_quantize_experts(gy, E, off, rows=False, cols=True, fmt=1), op, out=dw)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(24)
    for sizes in ([50, 50, 50, 50], [0, 200, 0, 0], [1, 2, 3, 4], [0, 0, 0, 0]):
        x.copy_(normal((T, C), 25 + sizes[1]))
        index.copy_(torch.randint(0, T, (S,), generator=g, dtype=torch.int32))
        off.copy_(torch.tensor(ends_of(sizes), dtype=torch.int32))
        for t in (y, dw):
            t.fill_(9.0)
        graph.replay()
        got = [y.clone(), dw.clone()]
        for t in (y, dw):
            t.fill_(9.0)
        step()
        assert torch.equal(y, got[0]) and torch.equal(dw, got[1])
        assert (y[sum(sizes):] == 9.0).all()


def test_calls_side_by_side(fq):
    """The same work on two streams at once, many times: results do not mix."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    jobs = []
    for k, s in enumerate(streams):
        x, w = normal((500, 512), 30 + k).cuda(), normal((3 * 512, 512), 32 + k).cuda()
        off = offsets_of([0, 120 + 40 * k, 300, 490])
        a, b = fq.fp8_quantize_experts(x, 3, off), fq.fp8_quantize_experts(w, 3)
        jobs.append((s, a, b, fq.fp8_experts_fprop(a, b, out=torch.zeros(500, 512, device="cuda"))))
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for s, a, b, _ in jobs:
            with torch.cuda.stream(s):
                outs.append(fq.fp8_experts_fprop(a, b, out=torch.zeros(500, 512, device="cuda")))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, jobs[i % 2][3])


def test_large_operands(fq):
    """More bytes and more results than 32 bits count, checked in a few rows."""
    S, C, N, E, T = 600_000, 4096, 4096, 3, 500
    x = normal((T, C), 40)
    index = (torch.arange(S, dtype=torch.int32) * 7) % T
    ends = [0, 1000, 1000, S - 5]
    off = offsets_of(ends)
    op = fq.fp8_quantize_experts(x.cuda(), E, off, index.cuda(), cols=True)
    some = [0, 999, 1000, 524_288, 524_289, S - 6]
    q, code = ref.mx_rows(f64(x[index[some].long()]), 0)
    np.testing.assert_array_equal(op.q[some].cpu().numpy(), q)
    blocks = fq.experts_blocks(S, E, True)
    first = ends[2] // 128 + 2
    col = 128 * first + S - 6 - 1000              # the last row's column
    tail = (S - 5 - 1000) % 32                    # rows of its last 32
    rows = index[S - 5 - tail:S - 5].long()
    want, _ = ref.mx_rows(f64(x[rows]).T, 0)
    np.testing.assert_array_equal(op.q_t[:, col - tail + 1:col + 1].cpu().numpy(), want)
    assert op.q_t.shape[1] == 128 * blocks
    w, _ = weights(fq, normal((E * N, C), 41, 0.05), E, transposed=False)
    y = torch.empty(S, N, dtype=BF16, device="cuda")
    fq.fp8_experts_fprop(op, w, out=y)
    values = ref.mx_values(q, code, 0)
    wv = list(ref.group_rows(arrays(w), ref.Groups([N * e for e in range(E + 1)], equal=True), 0))
    for i, r in enumerate(some):
        near(y[r:r + 1], values[i:i + 1], wv[0 if r < 1000 else 2], r)


def test_refusals(fq):
    x = torch.zeros(64, 64, dtype=BF16, device="cuda")
    off = offsets_of([0, 30, 64])
    op = fq.fp8_quantize_experts(x, 2, off)
    w = fq.fp8_quantize_experts(x, 2)
    bad = [lambda: fq.fp8_quantize_experts(x, 3),                               # 64 rows do not divide by 3
           lambda: fq.fp8_quantize_experts(x, 2, off.long()),
           lambda: fq.fp8_quantize_experts(x, 3, off),
           lambda: fq.fp8_quantize_experts(x, 2, off, index=off.long()),
           lambda: fq.fp8_quantize_experts(x, 2, off, rows=False),
           lambda: fq.fp8_quantize_experts(x, 2, off, cols=True, out=op),      # no storage for it
           lambda: fq.fp8_quantize_experts(x, 1025, offsets_of([0] * 1026)),
           lambda: fq.ExpertsOperand(64, 64, 2, 0, off, x, None),
           lambda: fq.fp8_experts_fprop(op, w, out=torch.zeros(64, 64, device="cuda"))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: fq.fp8_quantize_experts(x[:, :40], 2, off),               # cols % 16
              lambda: fq.fp8_quantize_experts(x, 2, off, fmt=7),
              lambda: fq.fp8_experts_fprop(op, op),                            # weights are equal groups
              lambda: fq.fp8_experts_dgrad(op, w),                             # not transposed, other sizes
              lambda: fq.fp8_experts_wgrad(op, op),
              lambda: fq.fp8_experts_fprop(op, fq.fp8_quantize_experts(x, 4))):
        with pytest.raises(fq.Fp8qError):
            f()

"""The experts' operators where calls follow one another closely, and at operands,
offsets and sizes that test_gpu_experts.py does not reach."""
import numpy as np
import pytest
import torch

import experts_reference as ref
from test_gpu_experts import BF16, FP32, MARK, arrays, ends_of, f64, fq, marked, near, normal, offsets_of, operand, weights  # noqa: F401

pytestmark = pytest.mark.gpu


def test_products_back_to_back(fq):
    """Launches that are set up while the one before them ends, each with another
    layout of shared memory, tiles from none to many a CTA pair: whatever a CTA
    still sent to its peer would land in the next one's barriers."""
    jobs = []
    for k, (sizes, N, K) in enumerate([([300, 0, 5, 140], 272, 400), ([1, 0, 0, 130], 1040, 144), ([600], 4112, 256),
                                       ([40] * 8, 144, 528), ([0, 2, 0, 3], 272, 4112)]):
        x, w, g = normal((sum(sizes), K), 60 + k), normal((len(sizes) * N, K), 70 + k, 0.05), normal((sum(sizes), N), 80 + k)
        xo, _ = operand(fq, x, sizes, 3, 0)
        go, _ = operand(fq, g, sizes, 3, 1)
        go = fq.ExpertsOperand(go.rows, go.cols, go.groups, 1, xo.offsets, go.q, go.q_scales, go.q_t, go.qt_scales)
        wo, _ = weights(fq, w, len(sizes))
        for out in (BF16, FP32):
            new = lambda *s: torch.full(s, 3.0, dtype=out, device="cuda")
            jobs += [(fq.fp8_experts_fprop, xo, wo, new(xo.rows, N)), (fq.fp8_experts_dgrad, go, wo, new(xo.rows, K)),
                     (fq.fp8_experts_wgrad, go, xo, new(len(sizes), N, K))]
    want = []
    for f, a, b, out in jobs:
        f(a, b, out=out)
        torch.cuda.synchronize()
        want.append(out.clone())
    order = np.random.default_rng(61)
    for _ in range(100):
        picked = order.permutation(len(jobs))
        for i in picked:
            f, a, b, out = jobs[i]
            f(a, b, out=out)
        for i in picked:
            assert torch.equal(jobs[i][3], want[i])
    assert fq.device_status() == fq.OK


@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("T", [0, 70])
def test_no_rows(fq, ragged, T):
    """A rank whose experts got no token: every call serves, dw is zero."""
    E, N, K = 4, 48, 80
    off = offsets_of([0] * (E + 1)) if ragged else None
    index = torch.empty(0, dtype=torch.int32, device="cuda")
    w, _ = weights(fq, normal((E * N, K), 90), E)
    for out in (BF16, FP32):
        x = fq.fp8_quantize_experts(normal((T, K), 91).cuda(), E, off, index, cols=True)
        g = fq.fp8_quantize_experts(normal((T, N), 92).cuda(), E, off, index, rows=True, cols=True, fmt=fq.E5M2)
        assert x.q.shape == (0, K)
        assert fq.fp8_experts_fprop(x, w, out_dtype=out).shape == (0, N)
        assert fq.fp8_experts_dgrad(g, w, out_dtype=out).shape == (0, K)
        dw = torch.full((E, N, K), 5.0, dtype=out, device="cuda")
        assert (fq.fp8_experts_wgrad(g, x, out=dw) == 0).all()
    if T == 0:   # without an index the operand's rows are x's
        x = fq.fp8_quantize_experts(torch.empty(0, K, device="cuda"), E, off, cols=True)
        assert fq.fp8_experts_fprop(x, w).shape == (0, N)


def test_no_rows_in_a_graph(fq):
    E, N, K = 3, 32, 64
    off = offsets_of([0] * (E + 1))
    x = fq.fp8_quantize_experts(torch.empty(0, K, device="cuda"), E, off, cols=True)
    g = fq.fp8_quantize_experts(torch.empty(0, N, device="cuda"), E, off, cols=True)
    dw = torch.full((E, N, K), 5.0, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.fp8_quantize_experts(torch.empty(0, K, device="cuda"), E, off, cols=True, out=x)
        fq.fp8_experts_wgrad(g, x, out=dw)
    graph.replay()
    assert (dw == 0).all()


def test_a_block_of_no_tokens():
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("experts_mxfp8", os.path.join(root, "examples", "experts_mxfp8.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.ExpertsBlock(128, 64, 8, 2)
    x = torch.empty(0, 128, dtype=BF16, device="cuda")
    out, saved = block.forward(x, x.clone())
    assert out.shape == x.shape
    dx, *grads = block.backward(out, saved)
    assert dx.shape == x.shape
    for d, w in zip(grads, (block.norm, block.router, block.up, block.down)):
        assert d.shape == w.shape and (d == 0).all()


@pytest.mark.parametrize("out", [BF16, FP32])
def test_gradient_of_operands_in_other_groups(fq, out):
    """g cast under another route's offsets: NaN where a group is not the same rows
    in both, in every order with groups that are, and empty ones; never another's sum."""
    S, N, K = 400, 272, 528
    ends = [0, 100, 130, 130, 130, 260, 261, 400]
    others = [[0, 100, 130, 130, 130, 260, 261, 400], [0, 100, 129, 130, 130, 260, 261, 400], [0, 0, 130, 130, 131, 260, 261, 390],
              [1, 100, 130, 130, 130, 260, 261, 400], [0] * 8, [-5, 100, 130, 130, 130, 260, 261, 400]]
    E, off = len(ends) - 1, offsets_of(ends)
    g, x = normal((S, N), 93, 0.1).cuda(), normal((S, K), 94).cuda()
    xo = fq.fp8_quantize_experts(x, E, off, rows=False, cols=True)
    want = fq.fp8_experts_wgrad(fq.fp8_quantize_experts(g, E, off, rows=False, cols=True, fmt=1), xo, out_dtype=out)
    for other in others:
        go = marked(fq, S, N, E, 1, offsets_of(other), by_rows=False)
        fq.fp8_quantize_experts(g, E, go.offsets, rows=False, cols=True, fmt=1, out=go)
        dw = torch.full((E, N, K), 5.0, dtype=out, device="cuda")
        fq.fp8_experts_wgrad(go, xo, out=dw)
        for e in range(E):
            if ends[e:e + 2] == [max(0, o) for o in other[e:e + 2]]:   # below 0 is 0
                assert torch.equal(dw[e], want[e]), (other, e)
            else:
                assert dw[e].isnan().all(), (other, e)
    torch.cuda.synchronize()
    assert fq.device_status() == fq.OK


def test_storage_under_a_view_of_its_offsets(fq):
    x, off = normal((60, 64), 95).cuda(), offsets_of([0, 20, 60])
    want = fq.fp8_quantize_experts(x, 2, off, cols=True)
    op = marked(fq, 60, 64, 2, 0, off)
    fq.fp8_quantize_experts(x, 2, off[:], cols=True, out=op)
    assert torch.equal(op.q, want.q)
    for other in (off.clone(), None):
        with pytest.raises(ValueError):
            fq.fp8_quantize_experts(x, 2, other, cols=True, out=op)


NONE = [[0, 50, 20, 70], [-5, 10, 90, 4000], [0, 70, 70, 2 ** 31 - 1], [60, 10, 0, 0], [-(2 ** 31), -1, 0, 12], [70, 70, 70, 70],
        [2 ** 31 - 1, 0, 2 ** 31 - 1, 0]]


@pytest.mark.parametrize("bad", NONE)
@pytest.mark.parametrize("scale,N,K", [(1, 272, 4112), (1, 4096, 272), (1, 272, 144), (10, 272, 144)])
@pytest.mark.parametrize("out", [BF16, FP32])
def test_offsets_that_are_none_in_every_kernel(fq, bad, scale, N, K, out):
    """Few rows, whose contraction (4112 of fprop, 4096 of dgrad) is split over a
    cluster, and tiles 256 and 128 wide: nothing is written beside the result, and offsets that are brought into
    [0, S] serve as those they become."""
    S, E = 70 * scale, 3
    off = offsets_of([max(-(2 ** 31), min(2 ** 31 - 1, b * scale)) for b in bad])
    inside = off.clamp(0, S)
    w, _ = weights(fq, normal((E * N, K), 96, 0.05), E)
    for f, cols, wide in ((fq.fp8_experts_fprop, K, N), (fq.fp8_experts_dgrad, N, K)):
        x = normal((S, cols), 97).cuda()
        got = []
        for o in (off, inside):
            op = marked(fq, S, cols, E, 0, o, transposed=False)
            fq.fp8_quantize_experts(x, E, o, out=op)
            result = torch.full((3, S, wide), 7.0, dtype=out, device="cuda")
            f(op, w, out=result[1])
            assert (result[0] == 7.0).all() and (result[2] == 7.0).all()
            got.append(result[1])
        ends = inside.tolist()
        if ends == sorted(ends):
            assert torch.equal(*got)
            assert (got[0][ends[-1]:] == 7.0).all() and (got[0][:ends[0]] == 7.0).all()
            assert (got[0][ends[0]:ends[-1]] != 7.0).any(dim=1).all()
    torch.cuda.synchronize()
    assert fq.device_status() == fq.OK


def test_large_input_gradient(fq):
    """More results than 32 bits count, checked in a few rows."""
    S, N, K, E, T = 600_000, 128, 4096, 3, 500
    g = normal((T, N), 98)
    index = (torch.arange(S, dtype=torch.int32) * 7) % T
    ends = [0, 1000, 1000, S - 5]
    op = fq.fp8_quantize_experts(g.cuda(), E, offsets_of(ends), index.cuda(), fmt=fq.E5M2)
    w, groups = weights(fq, normal((E * N, K), 99, 0.05), E, by_rows=False)
    dx = torch.full((S, K), 3.0, dtype=BF16, device="cuda")
    fq.fp8_experts_dgrad(op, w, out=dx)
    some = [0, 999, 1000, 524_287, 524_288, 524_289, S - 6]
    values = ref.mx_values(*ref.mx_rows(f64(g[index[some].long()]), 1), 1)
    wv = list(ref.group_cols(arrays(w), groups, 0))
    for i, r in enumerate(some):
        near(dx[r:r + 1], values[i:i + 1], wv[0 if r < 1000 else 2], r)
    assert (dx[S - 5:] == 3.0).all()


@pytest.mark.parametrize("out", [BF16, FP32])
def test_large_weight_gradient(fq, out):
    """More results than 32 bits count, checked in a few groups."""
    E, N, K = 256, 2048, 4128
    sizes = [i % 3 for i in range(E)]
    g, x = normal((sum(sizes), N), 100, 0.1), normal((sum(sizes), K), 101)
    go, groups = operand(fq, g, sizes, 2, 1, by_rows=False)
    xo, _ = operand(fq, x, sizes, 2, 0, by_rows=False)
    dw = torch.full((E, N, K), 5.0, dtype=out, device="cuda")
    assert dw.numel() > 2 ** 31
    fq.fp8_experts_wgrad(go, xo, out=dw)
    gv, xv = list(ref.group_cols(arrays(go), groups, 1)), list(ref.group_cols(arrays(xo), groups, 0))
    for e in (1, 127, 253, 254):
        near(dw[e], gv[e], xv[e], e)
    empty = torch.tensor([e for e in range(E) if sizes[e] == 0], device="cuda")
    assert all((dw[e] == 0).all() for e in empty.tolist())

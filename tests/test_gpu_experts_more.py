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

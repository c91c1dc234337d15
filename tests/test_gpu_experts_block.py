"""The example's block of experts, norm to combination and back, as a user would
run it: against fp32, token by token, and captured into a graph."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location(
        "experts_mxfp8", os.path.join(ROOT, "examples", "experts_mxfp8.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def inputs(tokens, hidden, n, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16() for _ in range(n)]


@pytest.mark.parametrize("size", [(256, 128, 8, 2, 300), (208, 144, 12, 3, 77), (128, 64, 4, 1, 1),
                                  (512, 256, 64, 4, 1000)])
def test_forward_and_gradients_follow_fp32(ex, size):
    """An operand in E4M3 is off by half a step of at most 2^-4, 0.036 in the mean
    square, one in E5M2 by twice that, relative.  `out` has four E4M3 operands
    behind it, 0.08 in all with bf16's roundings: a cosine of 0.995.  A gradient
    has at most four E4M3 and two E5M2 ones and the 8-bit checkpoint, 0.036 sqrt(6
    + 8) = 0.14: 0.98."""
    hidden, inner, experts, top, tokens = size
    block = ex.ExpertsBlock(hidden, inner, experts, top)
    x, residual, dout = inputs(tokens, hidden, 3)
    out, saved = block.forward(x, residual)
    got = (out, *block.backward(dout, saved))
    want = ex.reference(block, x, residual, dout, saved[2])
    for name, a, b in zip(("out", "dx", "dnorm", "drouter", "dup", "ddown"), got, want):
        assert a.shape == b.shape and a.isfinite().all(), name
        if name == "drouter" and top == 1:   # p is 1 whatever the scores
            assert (a == 0).all()
        else:
            assert ex.cosine(a, b) > (0.995 if name == "out" else 0.98), name


def test_tokens_one_by_one_are_the_batch(ex):
    """The same operands for a token wherever it stands: sums in another order,
    and one rounding to bf16 of u, v and o each."""
    block = ex.ExpertsBlock(256, 160, 8, 2)
    x, residual = inputs(200, 256, 2)
    whole, saved = block.forward(x, residual)
    for i in (0, 17, 199):
        one, s1 = block.forward(x[i:i + 1], residual[i:i + 1])
        assert torch.equal(s1[2].experts[0], saved[2].experts[i])
        a, b = one.float()[0], whole.float()[i]
        assert (a - b).norm() <= 0.02 * b.norm()


def test_a_captured_step_follows_its_inputs(ex):
    """Forward and backward in one graph, replayed on other tokens, which other
    experts get: bit for bit what the eager step gives."""
    block = ex.ExpertsBlock(128, 64, 8, 2)
    x, residual, dout = inputs(150, 128, 3)

    def step():
        out, saved = block.forward(x, residual)
        return (out, *block.backward(dout, saved))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (5, 6):
        for t, new in zip((x, residual, dout), inputs(150, 128, 3, seed)):
            t.copy_(new)
        graph.replay()
        kept = [t.clone() for t in got]
        for a, b in zip(kept, step()):
            assert torch.equal(a, b)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """With another device current, as the calls see it, nothing is launched."""
    import scaled_quantize_fp8_warp_gb300 as fq
    x, w = torch.randn(64, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda")
    op, wop = (fq.fp8_quantize_experts(x, 2, rows=True, cols=True) for _ in range(2))
    rstd = fq.fp8_rmsnorm(x, w).rstd
    out, y, narrow = (torch.full(s, 7.0, device="cuda") for s in ((2, 64, 64), (64, 64), (64, 32)))
    torch.cuda.synchronize()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for f in (lambda: fq.fp8_rmsnorm(x, w, y=y.bfloat16()), lambda: fq.fp8_rmsnorm_backward(x, x, w, rstd),
              lambda: fq.fp8_quantize_experts(x, 2, cols=True), lambda: fq.fp8_experts_fprop(op, wop, out=narrow),
              lambda: fq.fp8_experts_dgrad(op, wop, out=y), lambda: fq.fp8_experts_wgrad(op, op, out=out)):
        with pytest.raises(ValueError, match="current device"):
            f()
    monkeypatch.undo()
    assert all((t == 7.0).all() for t in (out, y, narrow)) and fq.device_status() == fq.OK

"""The experts' operators where calls follow one another closely, and at operands,
offsets and sizes that test_gpu_experts.py does not reach."""
import numpy as np
import pytest
import torch

import experts_reference as ref
from test_gpu_experts import BF16, FP32, MARK, arrays, ends_of, f64, fq, near, normal, offsets_of, operand, weights  # noqa: F401

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

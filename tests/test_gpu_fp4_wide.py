"""Products and training steps of many tiles: 384- and 256-wide tiles on CTA
pairs, alone and grouped, with several tiles a pair and several K blocks a tile
-- the ring carried over a tile's end, the accumulator handed over, the slots of
scales used again -- over the whole result, against a 64-bit product of the
values the operands stand for."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32
# (M, N, K, output, tile): odd counts of 128-row tiles, last tiles of 16 to 272
# columns, last K blocks of 40, 96 and 256
SIZES = [(3967, 6032, 2600, BF, 384), (5000, 5776, 4192, BF, 384), (8192, 4096, 4096, BF, 384),
         (3967, 6032, 2600, F32, 256), (3967, 6031, 2600, BF, 256), (3967, 6040, 4192, BF, 256),
         (4100, 5003, 1056, F32, 256)]
STEPS = [(4000, 6032, 2608, BF, 384), (8192, 4096, 4096, BF, 384), (3967, 4100, 2605, F32, 256)]


@pytest.fixture(scope="module")
def fq():
    import scaled_quantize_fp8_warp_gb300 as fq
    yield fq
    assert fq.device_status() == fq.OK


def normal(shape, seed, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def check(fq, got, qa, qb, what):
    """Within (K / 64 + 12) 2^-23 of the sum of magnitudes (an accumulator that
    drops what lies below its last place once per step of 64, the tensor scales
    and a join) and the output's rounding, doubled for a tie."""
    a = fq.fp4_dequantize(qa, out_dtype=F32).double()
    b = fq.fp4_dequantize(qb, out_dtype=F32).double()
    want, mag = a @ b.T, a.abs() @ b.abs().T
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -23
    err = (got.double() - want).abs()
    bad = err > (qa.K / 64 + 12) * 2.0 ** -23 * mag + half * want.abs()
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), float(err.max()))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("size", SIZES)
def test_gemm_and_linear(fq, kind, size):
    M, N, K, out, _ = size
    x, w = normal((M, K), 1), normal((N, K), 2, 0.02)
    qx, qw = fq.fp4_quantize(x, kind)[0], fq.fp4_quantize(w, kind)[0]
    y = fq.fp4_gemm(qx, qw, out_dtype=out)
    check(fq, y, qx, qw, "gemm")
    assert torch.equal(y, fq.fp4_linear(x, qw, out_dtype=out))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", STEPS)
def test_training_step(fq, kind, dtype, size):
    M, N, K, out, _ = size
    x, w, g = normal((M, K), 3, 1.0, dtype), normal((N, K), 4, 0.02, dtype), normal((M, N), 5, 1e-3, dtype)
    y, dx, dw = fq.fp4_linear_train(x, w, g, kind, out_dtype=out)
    (qx, qxt), (qw, qwt), (qg, qgt) = (fq.fp4_quantize(t, kind, cols=True) for t in (x, w, g))
    check(fq, y, qx, qw, "y")
    check(fq, dx, qg, qwt, "dx")
    check(fq, dw, qgt, qxt, "dw")


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("size", [(1, 16, 33), (96, 64, 160), (200, 130, 257), (333, 650, 1031)])
def test_training_step_from_fp32(fq, kind, out, size):
    M, N, K = size
    x, w, g = normal((M, K), 6, 1.0, F32), normal((N, K), 7, 0.02, F32), normal((M, N), 8, 1e-3, F32)
    y, dx, dw = fq.fp4_linear_train(x, w, g, kind, out_dtype=out)
    (qx, qxt), (qw, qwt), (qg, qgt) = (fq.fp4_quantize(t, kind, cols=True) for t in (x, w, g))
    check(fq, y, qx, qw, "y")
    check(fq, dx, qg, qwt, "dx")
    check(fq, dw, qgt, qxt, "dw")


def test_these_sizes_run_on_the_tiles_they_are_meant_for():
    script = f"""
import sys, torch
import scaled_quantize_fp8_warp_gb300 as fq
from torch import bfloat16, float32
for kind in (0, 1):
    for M, N, K, out, _ in {[(m, n, k, o, t) for m, n, k, o, t in SIZES]!r}:
        a, b = (fq.fp4_quantize(torch.zeros((r, K), dtype=bfloat16, device="cuda"), kind)[0] for r in (M, N))
        print("===", "gemm", M, N, K, file=sys.stderr, flush=True)
        fq.fp4_gemm(a, b, out_dtype=out)
    for M, N, K, out, _ in {[(m, n, k, o, t) for m, n, k, o, t in STEPS]!r}:
        x, w, g = (torch.zeros(s, dtype=bfloat16, device="cuda") for s in ((M, K), (N, K), (M, N)))
        print("===", "train", M, N, K, file=sys.stderr, flush=True)
        fq.fp4_linear_train(x, w, g, kind, out_dtype=out)
torch.cuda.synchronize()
""".replace("torch.bfloat16", "bfloat16").replace("torch.float32", "float32")
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, env=dict(os.environ, FP8Q_LOG="1"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    seen = {}
    for line in r.stderr.splitlines():
        if line.startswith("=== "):
            now = seen.setdefault(line[4:], [])
        elif "launch fp4 gemm_pair_kernel" in line or "launch fp4 split_kernel" in line:
            now.append(line)
    for sort, sizes in (("gemm", SIZES), ("train", STEPS)):
        for M, N, K, _, tile in sizes:
            lines = seen[f"{sort} {M} {N} {K}"]
            same = [t for t in sizes if t[:3] == (M, N, K)]
            assert len(lines) == 2 * len(same) * (1 if sort == "gemm" else 3), lines
            assert any(f"tile 256x{tile}" in s for s in lines), lines
            assert all("gemm_pair_kernel" in s and (sort == "gemm" or "grouped" in s) for s in lines), lines
            if len(same) == 1:
                assert all(f"tile 256x{tile}" in s for s in lines), lines

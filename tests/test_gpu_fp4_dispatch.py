"""How the few-row product divides its work, read from the launch log of a
child process (the switch is read once per process)."""
import os
import re
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = r"""
import sys, torch
import scaled_quantize_fp8_warp_gb300 as fq
fq.load_library()
def weight(N, K):
    rows = torch.zeros((N, (K + 31) // 32 * 16), dtype=torch.uint8, device="cuda")
    return fq.Fp4Operand(rows, torch.full((fq.fp4_scale_bytes(fq.MXFP4, N, K),), 127, dtype=torch.uint8, device="cuda"),
                         fq.MXFP4, K)
def mark(*what):
    print("===", *what, file=sys.stderr, flush=True)
"""


def logged(body):
    """{mark: its log lines} of a child that runs `body`."""
    r = subprocess.run([sys.executable, "-c", SETUP + body + "\ntorch.cuda.synchronize()\nassert fq.device_status() == 0\n"],
                       cwd=ROOT, env=dict(os.environ, FP8Q_LOG="1"), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out, now = {}, None
    for line in r.stderr.splitlines():
        if line.startswith("==="):
            now = out.setdefault(line[4:], [])
        elif now is not None:
            now.append(line)
    return out


def test_the_split_of_long_k_depends_on_the_tiles_alone():
    """With K long enough for four blocks a CTA whatever the split, tiles that
    run at once do so at any K; more tiles never take a larger split."""
    log = logged(r"""
for N in range(256, 12289, 256):
    for K in (8192, 12288, 14336, 16384):
        w, x = weight(N, K), torch.zeros((13, K), dtype=torch.bfloat16, device="cuda")
        mark(N, K)
        fq.fp4_linear(x, w)
""")
    split = {}
    for key, lines in log.items():
        N, K = map(int, key.split())
        (line,) = [s for s in lines if "split_kernel" in s]
        split.setdefault(N, set()).add(int(re.search(r"split (\d+)", line).group(1)))
    assert len(split) == 48 and all(len(s) == 1 for s in split.values()), split
    order = [max(split[N]) for N in sorted(split)]
    assert order == sorted(order, reverse=True)
    assert order[0] == 8 and order[-1] > 1


def test_a_training_step_shares_a_launch_only_where_one_is_saved():
    """By the times the choice goes by: three products that differ little go
    together; where one or both of the others belong on CTA pairs by more than
    a launch in all, none of the others is moved."""
    log = logged(r"""
for M, N, K in ((128, 128, 4096), (128, 1024, 16384), (200, 200, 16384)):
    x, w, g = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((M, K), (N, K), (M, N)))
    mark(M, N, K)
    fq.fp4_linear_train(x, w, g, fq.MXFP4)
""")
    kernels = {k: [("split" if "split_kernel" in s else "pair", "grouped" in s) for s in lines if "launch fp4" in s
                   and ("split_kernel" in s or "gemm_pair_kernel" in s)] for k, lines in log.items()}
    assert kernels["128 128 4096"] == [("split", True)] * 3
    for k in ("128 1024 16384", "200 200 16384"):
        assert kernels[k] == [("split", False), ("pair", True), ("pair", True)], kernels[k]

"""With FP8Q_LOG=1 the norm's and the experts' calls print a line of their own
and one for each kernel they launch, with its grid; and the rules that choose a
kernel (a child process: the switch is read once per process)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys, torch
import scaled_quantize_fp8_warp_gb300 as fq
fq.load_library()
def mark(name):
    print("=== " + name, file=sys.stderr, flush=True)
x = torch.randn(300, 512, device="cuda", dtype=torch.bfloat16)
w = torch.ones(512, device="cuda")
off = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
mark("norm")
n = fq.fp8_rmsnorm(x, w, x.clone())
mark("norm odd")
fq.fp8_rmsnorm(x[:, 1:200], w[:199], scaling=fq.SCALE_ROW)
mark("norm long")
long = torch.randn(3, 16400, device="cuda")
m = fq.fp8_rmsnorm(long, torch.ones(16400, device="cuda"))
mark("norm backward")
fq.fp8_rmsnorm_backward(x, n.h, w, n.rstd)
mark("norm backward long")
fq.fp8_rmsnorm_backward(long, long, torch.ones(16400, device="cuda"), m.rstd)
mark("cast")
a = fq.fp8_quantize_experts(x, 2, off(0, 100, 300), cols=True)
mark("weights")
b = fq.fp8_quantize_experts(torch.randn(2 * 256, 512, device="cuda"), 2, cols=True)
mark("fprop")
fq.fp8_experts_fprop(a, b)
mark("fprop fp32")
fq.fp8_experts_fprop(a, b, out_dtype=torch.float32)
mark("few rows")
c = fq.fp8_quantize_experts(torch.randn(5, 4096, device="cuda"), 2, off(0, 2, 5))
d = fq.fp8_quantize_experts(torch.randn(2 * 256, 4096, device="cuda"), 2)
fq.fp8_experts_fprop(c, d)
mark("narrow")
e = fq.fp8_quantize_experts(x, 8, off(*range(0, 360, 40)))
f = fq.fp8_quantize_experts(torch.randn(8 * 256, 512, device="cuda"), 8)
fq.fp8_experts_fprop(e, f)
mark("wgrad")
g = fq.fp8_quantize_experts(torch.randn(300, 256, device="cuda"), 2, a.offsets, cols=True, fmt=fq.E5M2)
fq.fp8_experts_wgrad(g, a)
mark("dgrad")
fq.fp8_experts_dgrad(g, b)
mark("end")
torch.cuda.synchronize()
assert fq.device_status() == 0
"""

EXPECT = {
    "norm": ["fp8_rmsnorm 300x512 residual=1 y=1 q=1", "launch norm forward_kernel bf16, 128 threads x 1 chunks a row, grid "],
    "norm odd": ["fp8_rmsnorm 300x199", "forward_kernel bf16 element by element, 32 threads"],
    "norm long": ["launch norm forward_long_kernel fp32, grid 3"],
    "norm backward": ["fp8_rmsnorm_backward 300x512", "launch norm backward_kernel bf16, 128 threads", "launch norm join_kernel"],
    "norm backward long": ["launch norm columns_kernel, grid 65 x 3", "launch norm backward_long_kernel fp32, grid 3"],
    "cast": ["fp8_quantize_experts 300 rows of 300x512 E=2 q=1 qt=1", "launch experts cast_kernel bf16, "],
    "weights": ["fp8_quantize_experts 512 rows of 512x512 E=2", "launch experts cast_kernel fp32, "],
    "fprop": ["fp8_experts_fprop S=300 N=256 K=512 E=2", "launch experts product_kernel, 2 groups, tile 256x256, grid "],
    "fprop fp32": ["product_kernel, 2 groups, tile 256x128"],
    "few rows": ["fp8_experts_fprop S=5", "launch experts split_product_kernel, 2 groups, K over 8 CTAs, grid 32"],
    "narrow": ["product_kernel, 8 groups, tile 256x128"],
    "wgrad": ["fp8_experts_wgrad S=300 N=256 K=512 E=2", "product_kernel, 2 groups, tile 256x256"],
    "dgrad": ["fp8_experts_dgrad S=300 N=256 K=512 E=2", "product_kernel, 2 groups, tile 256x256"],
}


def test_every_call_and_launch_prints_a_line():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=dict(os.environ, FP8Q_LOG="1"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    sections, cur = {}, None
    for line in r.stderr.splitlines():
        if line.startswith("=== "):
            cur = sections.setdefault(line[4:], [])
        elif cur is not None and line.startswith("[fp8q]"):
            cur.append(line)
    for name, needles in EXPECT.items():
        text = "\n".join(sections.get(name, []))
        for n in needles:
            assert n in text, f"{name}: '{n}' not in:\n{text}"

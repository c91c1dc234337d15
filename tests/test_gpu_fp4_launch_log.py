"""With FP8Q_LOG=1 the 4-bit and activation calls print a line of their own and
one for each kernel they launch, with its grid (a child process: the switch is
read once per process)."""
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
x = torch.randn(512, 256, device="cuda", dtype=torch.bfloat16)
w = torch.randn(1024, 256, device="cuda", dtype=torch.bfloat16)
odd = torch.randn(40, 100, device="cuda")[:, 1:98]
def mark(name):
    print("=== " + name, file=sys.stderr, flush=True)
mark("amax")
a = fq.fp4_amax(odd)
mark("cast")
qw, _ = fq.fp4_quantize(w, fq.NVFP4, amax=fq.fp4_amax(w))
mark("odd cast")
fq.fp4_quantize(odd, fq.NVFP4, cols=True, amax=a)
mark("empty cast")
fq.fp4_quantize(odd[:, :0], fq.NVFP4, amax=a)
qx, _ = fq.fp4_quantize(x, fq.NVFP4)
mark("dequantize")
fq.fp4_dequantize(qx)
mark("gemm")
fq.fp4_gemm(qx, qw)
mark("few rows")
fq.fp4_linear(x[:5], qw)
mark("linear")
fq.fp4_linear(x, qw)
mark("large gemm")
big = torch.zeros(8192, 512, device="cuda", dtype=torch.bfloat16)
qb, _ = fq.fp4_quantize(big, fq.MXFP4)
fq.fp4_gemm(qb, qb)
mark("train")
fq.fp4_linear_train(x, w, torch.zeros(512, 1024, device="cuda", dtype=torch.bfloat16), fq.NVFP4)
mark("act forward")
_, kept = fq.fp8_act_forward(fq.ACT_SILU, x, x)
mark("act backward")
fq.fp8_act_backward(fq.ACT_SILU, kept, x)
mark("odd act")
fq.fp8_act_forward(fq.ACT_GELU, odd)
mark("end")
torch.cuda.synchronize()
assert fq.device_status() == 0
"""

EXPECT = {
    "amax": ["fp4_amax 40x97", "launch fp4 amax_rows_kernel fp32 input, 40x97, grid "],
    "cast": ["fp4_quantize 1024x256 kind=1", "launch fp4 quantize_kernel kind 1 bf16 input, 1 matrices", "grid 16"],
    "odd cast": ["fp4_quantize 40x97", "fp32 input element by element", "grid 1"],
    "empty cast": ["fp4_quantize 40x0", "launch fp4 global_kernel grid 1"],
    "dequantize": ["fp4_dequantize 512x256", "launch fp4 dequantize_kernel kind 1 bf16 output", "grid 1x128"],
    "gemm": ["fp4_gemm M=512 N=1024 K=256", "launch fp4 ", "_kernel 512x1024x256", "1 products", "grid "],
    "few rows": ["fp4_linear M=5 N=1024 K=256", "launch amax_kernel", "launch fp4 split_kernel 5x1024x256",
                 "quantising x", "in clusters of"],
    "linear": ["fp4_linear M=512", "launch fp4 quantize_kernel", "_kernel 512x1024x256"],
    "large gemm": ["launch fp4 gemm_pair_kernel 8192x8192x512 kind 0 tile 256x384", "in pairs"],
    "train": ["fp4_linear_train M=512 N=1024 K=256", "launch fp4 amax_group_kernel bf16 input, grid ",
              "launch fp4 quantize_kernel kind 1 bf16 input, 3 matrices", "512x256x1024", "1024x256x512"],
    "act forward": ["fp8_act_forward act=0 512x256 gated=1", "launch act forward_kernel act 0 bf16 gated", "grid "],
    "act backward": ["fp8_act_backward act=0 512x256", "launch act backward_kernel act 0 bf16 gated", "grid "],
    "odd act": ["fp8_act_forward act=1 40x97 gated=0", "forward_kernel act 1 fp32 element by element"],
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

"""A gated feed-forward layer in 4 bits, trained and then served.

    h = x W_up^T,  (u, v) = the halves of h,  a = silu(u) v,  y = a W_down^T

The products run in MXFP4 or NVFP4 (fp4_linear, fp4_gemm); what the activation
keeps for the backward pass is u and v in E4M3 under 1x128 tile scales
(fp8_act_forward, fp8_act_backward), a quarter of what fp32 activations or half
of what bf16 ones take.  Master weights stay in fp32.  Serving holds only the
4-bit weights and runs token by token.

Usage: python examples/feed_forward_4bit.py [--kind nvfp4] [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scaled_quantize_fp8_warp_gb300 as fq  # noqa: E402


class FeedForward4Bit:
    """One layer's weights (fp32 masters) with its forward and backward pass."""

    def __init__(self, hidden: int, ffn: int, kind: int, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        draw = lambda *s, scale: torch.randn(s, generator=g, device=device) * scale
        self.kind, self.ffn = kind, ffn
        self.w_up = draw(2 * ffn, hidden, scale=hidden ** -0.5)
        self.w_down = draw(hidden, ffn, scale=ffn ** -0.5)

    def forward(self, x):
        """x [T, hidden] bf16 -> y [T, hidden] bf16, and what backward needs:
        x and the weights in 4 bits the other way round, u and v in 8."""
        up, up_t = fq.fp4_quantize(self.w_up, self.kind, cols=True)
        down, down_t = fq.fp4_quantize(self.w_down, self.kind, cols=True)
        x4, x4_t = fq.fp4_quantize(x, self.kind, cols=True)
        h = fq.fp4_gemm(x4, up)
        a, kept = fq.fp8_act_forward(fq.ACT_SILU, h[:, :self.ffn], h[:, self.ffn:])
        y = fq.fp4_linear(a, down)
        return y, (x4_t, up_t, down_t, kept)

    def backward(self, dy, saved):
        """dy [T, hidden] bf16 -> (dx bf16, dW_up fp32, dW_down fp32)."""
        x4_t, up_t, down_t, kept = saved
        dy4, dy4_t = fq.fp4_quantize(dy, self.kind, cols=True)
        da = fq.fp4_gemm(dy4, down_t)
        dh = torch.empty((dy.shape[0], 2 * self.ffn), dtype=dy.dtype, device=dy.device)
        _, _, a = fq.fp8_act_backward(fq.ACT_SILU, kept, da, want_a=True,
                                      du=dh[:, :self.ffn], dv=dh[:, self.ffn:])
        _, a4_t = fq.fp4_quantize(a, self.kind, rows=False, cols=True)
        dw_down = fq.fp4_gemm(dy4_t, a4_t, out_dtype=torch.float32)
        dh4, dh4_t = fq.fp4_quantize(dh, self.kind, cols=True)
        dw_up = fq.fp4_gemm(dh4_t, x4_t, out_dtype=torch.float32)
        return fq.fp4_gemm(dh4, up_t), dw_up, dw_down

    def serving(self, x_calibration):
        """A function of one batch of tokens that holds the weights in 4 bits
        and, for NVFP4, the input scales found on a calibration batch."""
        up, _ = fq.fp4_quantize(self.w_up, self.kind)
        down, _ = fq.fp4_quantize(self.w_down, self.kind)
        h = fq.fp4_gemm(fq.fp4_quantize(x_calibration, self.kind)[0], up)
        a, _ = fq.fp8_act_forward(fq.ACT_SILU, h[:, :self.ffn], h[:, self.ffn:])
        x_amax, a_amax = (fq.fp4_amax(x_calibration), fq.fp4_amax(a)) if self.kind == fq.NVFP4 \
            else (None, None)

        def run(x):
            h = fq.fp4_linear(x, up, x_amax=x_amax)
            a, _ = fq.fp8_act_forward(fq.ACT_SILU, h[:, :self.ffn], h[:, self.ffn:])
            return fq.fp4_linear(a, down, x_amax=a_amax)
        return run


def reference(layer: FeedForward4Bit, x, dy):
    """The same layer and its gradients in fp32."""
    w_up, w_down = (w.clone().requires_grad_() for w in (layer.w_up, layer.w_down))
    x = x.float().requires_grad_()
    u, v = (x @ w_up.t()).chunk(2, dim=1)
    y = (torch.nn.functional.silu(u) * v) @ w_down.t()
    y.backward(dy.float())
    return y.detach(), x.grad, w_up.grad, w_down.grad


def cosine(a, b):
    return float(torch.nn.functional.cosine_similarity(a.double().flatten(), b.double().flatten(), dim=0))


def train(layer: FeedForward4Bit, steps: int, tokens: int, seed: int = 1, lr: float = 2e-3):
    """Fits the layer to a teacher of its own shape with Adam; the losses."""
    teacher = FeedForward4Bit(layer.w_down.shape[0], layer.ffn, layer.kind, seed=seed + 100)
    opt = torch.optim.Adam([layer.w_up, layer.w_down], lr=lr)
    g = torch.Generator(device="cuda").manual_seed(seed)
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, layer.w_down.shape[0]), generator=g, device="cuda").bfloat16()
        u, v = (x.float() @ teacher.w_up.t()).chunk(2, dim=1)
        target = (torch.nn.functional.silu(u) * v) @ teacher.w_down.t()
        y, saved = layer.forward(x)
        err = y.float() - target
        losses.append(float(err.square().mean()))
        _, layer.w_up.grad, layer.w_down.grad = layer.backward((2 * err / err.numel()).bfloat16(),
                                                               saved)
        opt.step()
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--kind", choices=("mxfp4", "nvfp4"), default="nvfp4")
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--ffn", type=int, default=2048)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=60)
    args = ap.parse_args(argv)
    kind = fq.NVFP4 if args.kind == "nvfp4" else fq.MXFP4
    torch.manual_seed(0)
    layer = FeedForward4Bit(args.hidden, args.ffn, kind)
    x = torch.randn((args.tokens, args.hidden), device="cuda").bfloat16()
    dy = (torch.randn((args.tokens, args.hidden), device="cuda") * 1e-3).bfloat16()
    y, saved = layer.forward(x)
    got = (y, *layer.backward(dy, saved))
    for name, a, b in zip(("y", "dx", "dW_up", "dW_down"), got, reference(layer, x, dy)):
        print(f"{name:8s} cosine with fp32: {cosine(a, b):.4f}")
    kept = saved[3]
    held = sum(t.numel() * t.element_size() for t in (kept.u, kept.u_scales, kept.v, kept.v_scales))
    print(f"the activation keeps {held / 2 ** 20:.2f} MiB; bf16 would take "
          f"{2 * kept.u.numel() * 2 / 2 ** 20:.2f}")
    losses = train(layer, args.steps, args.tokens)
    print(f"{args.kind} training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {args.steps} steps")
    serve = layer.serving(x)
    one = torch.cat([serve(x[i:i + 1]) for i in range(8)])
    print(f"8 tokens one by one against the batch: cosine {cosine(one, serve(x)[:8]):.5f}")


if __name__ == "__main__":
    main()

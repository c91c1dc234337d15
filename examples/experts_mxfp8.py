"""A pre-norm feed-forward of experts in MXFP8, trained and served.

    h = x + residual,  y = norm(h),  scores = y W_router^T
    each token goes to its `top` best experts, with weights p = softmax of their scores
    o = sum over them of p (silu(u) v) W_down_e^T,  (u, v) the halves of y W_up_e^T
    out = h + o

The norm and its backward pass, the cast of the routed rows and the experts'
products are this library's (fp8_rmsnorm, fp8_quantize_experts,
fp8_experts_fprop / _dgrad / _wgrad), the activation keeps its inputs in 8 bits
(fp8_act_forward).  How many rows an expert gets is known on the device only:
nothing here waits for it, so a step can be captured into a CUDA graph.

Usage: python examples/experts_mxfp8.py [--experts 16] [--top 2] [--steps 40]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import scaled_quantize_fp8_warp_gb300 as fq  # noqa: E402


class Route:
    """Which expert every token goes to, and the rows in the experts' order:
    row r is token index[r]; choice j of token t is row place[t, j]."""

    def __init__(self, scores: torch.Tensor, top: int):
        E = scores.shape[1]
        self.experts = scores.topk(top, dim=1).indices
        flat = self.experts.reshape(-1)
        sorted_experts, order = torch.sort(flat, stable=True)
        self.index = torch.div(order, top, rounding_mode="floor").int()
        bounds = torch.arange(E + 1, device=scores.device)
        self.offsets = torch.searchsorted(sorted_experts, bounds).int()
        self.place = torch.empty_like(order).scatter_(0, order, torch.arange(len(order), device=order.device))
        self.place = self.place.view(-1, top)

    def weights(self, scores: torch.Tensor) -> torch.Tensor:
        return scores.gather(1, self.experts).softmax(dim=1)


class ExpertsBlock:
    """The weights (fp32 masters) of one block with its forward and backward pass."""

    def __init__(self, hidden: int, inner: int, experts: int, top: int, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        draw = lambda *s, scale: torch.randn(s, generator=g, device=device) * scale
        self.inner, self.E, self.top = inner, experts, top
        self.norm = 1.0 + draw(hidden, scale=0.1)
        self.router = draw(experts, hidden, scale=hidden ** -0.5)
        self.up = draw(experts * 2 * inner, hidden, scale=hidden ** -0.5)
        self.down = draw(experts * hidden, inner, scale=inner ** -0.5)

    def forward(self, x, residual, route: Route | None = None):
        """x, residual [T, hidden] bf16 -> out [T, hidden] bf16, and what backward needs."""
        up = fq.fp8_quantize_experts(self.up, self.E, cols=True)
        down = fq.fp8_quantize_experts(self.down, self.E, cols=True)
        n = fq.fp8_rmsnorm(x, self.norm, residual=residual, scaling=None)
        scores = n.y.float() @ self.router.t()
        route = route if route is not None else Route(scores, self.top)
        p = route.weights(scores)
        y8 = fq.fp8_quantize_experts(n.y, self.E, route.offsets, route.index, cols=True)
        uv = fq.fp8_experts_fprop(y8, up)
        a, kept = fq.fp8_act_forward(fq.ACT_SILU, uv[:, :self.inner], uv[:, self.inner:])
        a8 = fq.fp8_quantize_experts(a, self.E, route.offsets, cols=True)
        o = fq.fp8_experts_fprop(a8, down)
        out = n.h.float() + (o[route.place].float() * p[..., None]).sum(dim=1)
        return out.bfloat16(), (n, scores, route, p, up, down, y8, kept, a8, o)

    def backward(self, dout, saved):
        """dout [T, hidden] bf16 -> (dx, dnorm, drouter, dup, ddown); dx is the
        gradient of x and of the residual."""
        n, scores, route, p, up, down, y8, kept, a8, o = saved
        E = self.E
        # every row's gradient is its token's, times its weight
        weight = torch.empty(o.shape[0], device=o.device).scatter_(0, route.place.reshape(-1), p.reshape(-1))
        do = (dout.float()[route.index.long()] * weight[:, None]).bfloat16()
        do8 = fq.fp8_quantize_experts(do, E, route.offsets, cols=True, fmt=fq.E5M2)
        da = fq.fp8_experts_dgrad(do8, down)
        ddown = fq.fp8_experts_wgrad(do8, a8, out_dtype=torch.float32)
        duv = torch.empty((do.shape[0], 2 * self.inner), dtype=dout.dtype, device=dout.device)
        fq.fp8_act_backward(fq.ACT_SILU, kept, da, du=duv[:, :self.inner], dv=duv[:, self.inner:])
        duv8 = fq.fp8_quantize_experts(duv, E, route.offsets, cols=True, fmt=fq.E5M2)
        dy = fq.fp8_experts_dgrad(duv8, up)[route.place].float().sum(dim=1)
        dup = fq.fp8_experts_wgrad(duv8, y8, out_dtype=torch.float32)
        # the router: p = softmax of the chosen scores
        dp = (o[route.place].float() * dout.float()[:, None]).sum(dim=2)
        chosen = p * (dp - (dp * p).sum(dim=1, keepdim=True))
        dscores = torch.zeros_like(scores).scatter_(1, route.experts, chosen)
        dy = dy + dscores @ self.router
        drouter = dscores.t() @ n.y.float()
        dx, dnorm = fq.fp8_rmsnorm_backward(dy.bfloat16(), n.h, self.norm, n.rstd, dresidual=dout)
        return dx, dnorm, drouter, dup.view_as(self.up), ddown.view_as(self.down)


def reference(block: ExpertsBlock, x, residual, dout, route: Route):
    """The same block and its gradients in fp32, for the same choice of experts."""
    leaves = [t.clone().float().requires_grad_() for t in (x, block.norm, block.router, block.up, block.down)]
    x, norm, router, up, down = leaves
    h = x + residual.float()
    y = torch.nn.functional.rms_norm(h, (h.shape[1],), norm, 1e-6)
    p = route.weights(y @ router.t())
    rows, bounds = y[route.index.long()], route.offsets.tolist()
    up, down = up.view(block.E, -1, up.shape[1]), down.view(block.E, -1, down.shape[1])
    o = []
    for e in range(block.E):
        u, v = (rows[bounds[e]:bounds[e + 1]] @ up[e].t()).chunk(2, dim=1)
        o.append((torch.nn.functional.silu(u) * v) @ down[e].t())
    out = h + (torch.cat(o)[route.place] * p[..., None]).sum(dim=1)
    out.backward(dout.float())
    return out.detach(), *(t.grad for t in leaves)


def cosine(a, b):
    return float(torch.nn.functional.cosine_similarity(a.double().flatten(), b.double().flatten(), dim=0))


def train(block: ExpertsBlock, steps: int, tokens: int, seed: int = 1, lr: float = 1e-3):
    """Fits the block to a dense teacher with Adam; the losses."""
    hidden = block.norm.shape[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher = torch.randn((hidden, hidden), generator=g, device="cuda") * hidden ** -0.5
    weights = [block.norm, block.router, block.up, block.down]
    opt = torch.optim.Adam(weights, lr=lr)
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
        none = torch.zeros_like(x)
        out, saved = block.forward(x, none)
        err = out.float() - x.float() - torch.tanh(x.float() @ teacher.t())
        losses.append(float(err.square().mean()))
        _, *grads = block.backward((2 * err / tokens).bfloat16(), saved)
        for w, d in zip(weights, grads):
            w.grad = d
        opt.step()
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--inner", type=int, default=256)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=40)
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    block = ExpertsBlock(args.hidden, args.inner, args.experts, args.top)
    x, residual, dout = (torch.randn((args.tokens, args.hidden), device="cuda").bfloat16() for _ in range(3))
    out, saved = block.forward(x, residual)
    got = (out, *block.backward(dout, saved))
    for name, a, b in zip(("out", "dx", "dnorm", "drouter", "dup", "ddown"), got,
                          reference(block, x, residual, dout, saved[2])):
        print(f"{name:8s} cosine with fp32: {cosine(a, b):.4f}")
    losses = train(block, args.steps, args.tokens)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {args.steps} steps")
    one = torch.cat([block.forward(x[i:i + 1], residual[i:i + 1])[0] for i in range(8)])
    print(f"8 tokens one by one against the batch: cosine {cosine(one, block.forward(x, residual)[0][:8]):.5f}")


if __name__ == "__main__":
    main()

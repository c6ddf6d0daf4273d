"""A mixture-of-experts layer trained on one MI355X with the library's
operators end to end:

    router -> token groups -> dispatch -> MXFP8 operands -> expert products
    -> combine (+ residual) -> loss, balance and z losses
    -> gradients back through combine, dispatch and router
    -> Muon update of the 3-D expert weights, quantized again next step

The group ends never leave the device.  The products themselves are plain
torch on the dequantized operands (the library has no grouped GEMM), each
expert over all rows and kept where the row is its own; gradients pass the
quantizers straight through.

    python examples/moe_train_step.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_quantization_moe_amd as mxq  # noqa: E402


class Route(torch.autograd.Function):
    """logits -> the slots' weights and the two losses; the rest of the route
    is handed over through ``box``."""

    @staticmethod
    def forward(ctx, logits, top_k, align, box):
        route = mxq.moe_route(logits, top_k, align=align)
        box.append(route)
        ctx.route = route
        ctx.save_for_backward(logits)
        return route.weights, route.losses

    @staticmethod
    def backward(ctx, grad_weights, grad_losses):
        (logits,) = ctx.saved_tensors
        return mxq.moe_route_backward(logits, ctx.route, grad_weights, grad_losses), None, None, None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, route):
        ctx.route = route
        return mxq.moe_dispatch(x, route)

    @staticmethod
    def backward(ctx, grad_xg):
        return mxq.moe_dispatch_backward(grad_xg, ctx.route), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, yg, weights, residual, route):
        ctx.route = route
        ctx.save_for_backward(yg)
        return mxq.moe_combine(yg, route, residual=residual)

    @staticmethod
    def backward(ctx, grad_y):
        (yg,) = ctx.saved_tensors
        grad_yg, grad_weights = mxq.moe_combine_backward(grad_y, yg, ctx.route)
        return grad_yg, grad_weights, grad_y, None


class QuantizeRows(torch.autograd.Function):
    """bf16 rows through MXFP8 (1 x 32 blocks) and back; straight-through gradient."""

    @staticmethod
    def forward(ctx, x):
        q, scales = mxq.quantize_mx_rowwise(x)
        factor = torch.exp2(scales.float() - 127.0).repeat_interleave(32, 1)
        return (q.float() * factor).to(x.dtype)

    @staticmethod
    def backward(ctx, grad):
        return grad


class QuantizeWeights(torch.autograd.Function):
    """Expert weights (E, N, K) through MXFP8 (32 x 1 blocks along N)."""

    @staticmethod
    def forward(ctx, w):
        q, scales = mxq.quantize_mx_3d_colwise(w)
        factor = torch.exp2(scales.float() - 127.0).repeat_interleave(32, 1)
        return (q.float() * factor).to(w.dtype)

    @staticmethod
    def backward(ctx, grad):
        return grad


def expert_products(xg, w, offs):
    """Row r of xg times its expert's (N, K) weights, transposed: (rows, N)."""
    rows = torch.arange(xg.shape[0], device=xg.device)
    expert = torch.searchsorted(offs, rows, right=True)
    y = torch.zeros(xg.shape[0], w.shape[1], dtype=xg.dtype, device=xg.device)
    for e in range(w.shape[0]):
        y = torch.where((expert == e)[:, None], xg @ w[e].t().contiguous(), y)
    return y


class MoeLayer:
    def __init__(self, width, hidden, experts, top_k, align=32):
        g = torch.Generator(device="cuda").manual_seed(1)
        new = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5)  # noqa: E731
        self.router = new(experts, width).requires_grad_()
        self.up = new(experts, hidden, width).to(torch.bfloat16).requires_grad_()
        self.down = new(experts, width, hidden).to(torch.bfloat16).requires_grad_()
        self.momentum = {n: torch.zeros_like(getattr(self, n), dtype=torch.float32) for n in ("up", "down")}
        self.workspace = {n: mxq.muon_workspace(*getattr(self, n).shape) for n in ("up", "down")}
        self.top_k, self.align = top_k, align

    def __call__(self, x):
        box = []
        weights, losses = Route.apply(x.float() @ self.router.t(), self.top_k, self.align, box)
        route = box[0]
        xg = QuantizeRows.apply(Dispatch.apply(x, route))
        h = torch.relu(expert_products(xg, QuantizeWeights.apply(self.up), route.offs))
        yg = expert_products(QuantizeRows.apply(h), QuantizeWeights.apply(self.down), route.offs)
        return Combine.apply(yg, weights, x, route), losses, route

    def update(self, lr, router_lr):
        with torch.no_grad():
            for name in ("up", "down"):
                w = getattr(self, name)
                m = self.momentum[name].mul_(0.9).add_(w.grad.float())
                # the usual scale of an orthogonal update: rms 0.2 per element
                scale = 0.2 * max(w.shape[1:]) ** 0.5
                w.sub_(lr * mxq.muon_orthogonalize(m, scale=scale, workspace=self.workspace[name]))
                w.grad = None
            self.router.sub_(router_lr * self.router.grad)
            self.router.grad = None


def train(steps=60, tokens=2048, width=256, hidden=512, experts=8, top_k=2, verbose=True):
    layer = MoeLayer(width, hidden, experts, top_k)
    g = torch.Generator(device="cuda").manual_seed(2)
    teacher = torch.randn(width, width, generator=g, device="cuda") * width ** -0.5
    history = []
    for step in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda")
        target = x + torch.relu(x @ teacher.t())
        y, losses, route = layer(x.to(torch.bfloat16))
        fit = (y.float() - target).square().mean()
        (fit + 1e-2 * losses[0] + 1e-3 * losses[1]).backward()
        layer.update(lr=2e-2 * (1 - step / steps), router_lr=0.1)
        history.append(torch.stack([fit.detach(), losses[0].detach(), route.counts.max().float()]))
    history = torch.stack(history).tolist()
    if verbose:
        for step in sorted({0, steps // 4, steps // 2, steps - 1}):
            fit, balance, most = history[step]
            print(f"step {step:4d}  fit {fit:.4f}  balance {balance:.4f}  fullest expert {most:.0f} of "
                  f"{tokens * top_k / experts:.0f} even")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps)

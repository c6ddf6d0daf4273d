"""A mixture-of-experts layer trained on one MI355X with the library's
operators end to end:

    router -> token groups -> dispatch -> MXFP8 operands -> expert products
    with the activation -> combine (+ residual) -> loss, balance and z losses
    -> gradients back through combine, products, dispatch and router
    -> Muon update of the 3-D expert weights, quantized again next step

The group ends never leave the device.  The products run on MXFP8 operands,
their gradients on the bf16 ones: gradients pass the quantizers straight
through.  ``MoeLayer.decode`` runs the trained layer for a few tokens.

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


class ExpertProducts(torch.autograd.Function):
    """Row r of x times its expert's (N, K) weights, transposed, on MXFP8
    operands with 1 x 32 blocks along K; then the activation."""

    @staticmethod
    def forward(ctx, x, w, offs, activation):
        q, scales = mxq.quantize_mx_rowwise(x)
        wq, wscales = mxq.quantize_mx_rowwise(w.view(-1, w.shape[2]))
        y, pre = mxq.moe_linear_mx(q, scales, wq.view(w.shape), wscales.view(*w.shape[:2], -1), offs,
                                   activation=activation, save_pre=True)
        ctx.activation = activation
        ctx.save_for_backward(x, w, offs, pre)
        return y

    @staticmethod
    def backward(ctx, grad_y):
        x, w, offs, pre = ctx.saved_tensors
        grad_x, grad_w, _ = mxq.moe_linear_backward(grad_y, x, w, offs, pre=pre, activation=ctx.activation,
                                                    need_x=ctx.needs_input_grad[0], need_w=ctx.needs_input_grad[1])
        return grad_x, grad_w, None, None


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
        h = ExpertProducts.apply(Dispatch.apply(x, route), self.up, route.offs, "relu")
        yg = ExpertProducts.apply(h, self.down, route.offs, "none")
        return Combine.apply(yg, weights, x, route), losses, route

    def decode(self, x):
        """The layer for up to 64 tokens, the weights as they are."""
        with torch.no_grad():
            return mxq.moe_layer(x, x.float() @ self.router.t(), self.up, self.down, self.top_k, activation="relu",
                                 gated=False, residual=x)

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
    few = x[:16].to(torch.bfloat16)
    off = torch.linalg.vector_norm(layer.decode(few).float() - layer(few)[0].float()).item()
    history = torch.stack(history).tolist()
    if verbose:
        print(f"16 tokens decoded with bf16 weights, {off:.3g} (2-norm) from the MXFP8 products")
        for step in sorted({0, steps // 4, steps // 2, steps - 1}):
            fit, balance, most = history[step]
            print(f"step {step:4d}  fit {fit:.4f}  balance {balance:.4f}  fullest expert {most:.0f} of "
                  f"{tokens * top_k / experts:.0f} even")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps)

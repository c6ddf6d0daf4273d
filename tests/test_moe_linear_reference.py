"""The products' 64-bit gradients against differences of the 64-bit forward."""
import pytest
import torch

import linear_reference as ref


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu"])
def test_gradients(name, gated):
    g = torch.Generator().manual_seed(7)
    rows, width, n, offs = 9, 5, 4, [3, 3, 8]
    wide = 2 * n if gated else n
    x, w, b, dy = (torch.randn(*s, generator=g, dtype=torch.float64)
                   for s in ((rows, width), (3, wide, width), (3, wide), (rows, n)))
    _, z, _ = ref.forward(x, w, offs, b, name, gated)
    dz = ref.grad_z(dy, z, name, gated)
    grads = ref.backward(dz, x, w, offs)
    for t, grad in zip((x, w, b), grads):
        for at in torch.randint(t.numel(), (6,), generator=g).tolist():
            flat = t.view(-1)
            old, h, vals = flat[at].item(), 1e-6, []
            for d in (h, -h):
                flat[at] = old + d
                vals.append((ref.forward(x, w, offs, b, name, gated)[0] * dy).sum().item())
            flat[at] = old
            # central differences in 64 bits: 1e-12 / 1e-6 of rounding, h^2 of curvature
            assert abs((vals[0] - vals[1]) / (2 * h) - grad.view(-1)[at].item()) < 1e-7

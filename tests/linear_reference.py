"""The experts' products from their definition in 64 bits, group by group, with
the magnitudes that bound a sum's rounding errors."""
from __future__ import annotations

import math

import torch


def act(z, name):
    """The activation and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z < 0, 0.0, z), (z > 0).to(z.dtype)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(z)
    return z * s, s * (1 + z * (1 - s))


def groups(offs, rows):
    ends = [rows] if offs is None else [min(max(int(v), 0), rows) for v in offs]
    return list(zip([0] + ends[:-1], ends))


def mx_values(q, scales):
    """What e4m3 codes and e8m0 scales along the last dim stand for."""
    one = torch.ones((), dtype=torch.float64, device=q.device)
    return q.double() * torch.ldexp(one, scales.int() - 127).repeat_interleave(32, -1)


def forward(x, w, offs, bias=None, name="none", gated=False, resid=None):
    """(y, z, size): size bounds the fp32 terms behind each y."""
    rows, wide = x.shape[0], w.shape[1]
    n = wide // 2 if gated else wide
    z, zsize = (torch.zeros(rows, wide, dtype=torch.float64, device=x.device) for _ in range(2))
    used = torch.zeros(rows, 1, dtype=torch.bool, device=x.device)
    for e, (lo, hi) in enumerate(groups(offs, rows)):
        if hi <= lo:
            continue
        z[lo:hi] = x[lo:hi] @ w[e].t()
        zsize[lo:hi] = x[lo:hi].abs() @ w[e].abs().t()
        if bias is not None:
            z[lo:hi] += bias[e].double()
            zsize[lo:hi] += bias[e].double().abs()
        used[lo:hi] = True
    a, slope = act(z[:, :n], name)
    # an error d of z is one of at most 1.13 d of the activation
    y, size = a, 1.13 * zsize[:, :n]
    if gated:
        y, size = a * z[:, n:], size * z[:, n:].abs() + a.abs() * zsize[:, n:]
    if resid is not None:
        y, size = y + resid.double(), size + resid.double().abs()
    return torch.where(used, y, 0.0), z, size


def grad_z(dy, z, name, gated):
    if name == "none" and not gated:
        return dy
    n = dy.shape[1]
    a, slope = act(z[:, :n], name)
    return torch.cat([dy * z[:, n:] * slope, dy * a], 1) if gated else dy * slope


def backward(dz, x, w, offs):
    """(grad_x, grad_w, grad_bias) of dz."""
    gx = torch.zeros_like(x)
    gw = torch.zeros_like(w)
    gb = torch.zeros(w.shape[:2], dtype=x.dtype, device=x.device)
    for e, (lo, hi) in enumerate(groups(offs, x.shape[0])):
        if hi > lo:
            gx[lo:hi] = dz[lo:hi] @ w[e]
            gw[e] = dz[lo:hi].t() @ x[lo:hi]
            gb[e] = dz[lo:hi].sum(0)
    return gx, gw, gb

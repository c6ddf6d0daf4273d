"""GELU far below zero, where its value is the small tail of the normal
distribution: right relative to that value, in every kernel that applies it."""
import math

import pytest
import torch

import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = 2.0 ** -8
# The exponent x^2 / 2 reaches 72 (104 in base 2), and its rounding to fp32 (three
# operations, 2^-24 each) is a relative error of its exponential of
# 104 ln 2 * 3 * 2^-24 = 1.3e-5; the other dozen roundings and a fit of 2e-7 are less
# than 3e-6 together.
TAIL = 1.6e-5


def points(lo, hi):
    """Every bf16 from lo to hi."""
    v = torch.arange(0, 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = torch.cat([-v.flip(0), v])
    v = v[(v >= lo) & (v <= hi)]
    return v.unique().to(DEV)


def value(z):
    return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))


def slope(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def grid(v, rows):
    """The points over `rows` rows and 64 columns, repeated as needed."""
    at = torch.arange(rows * 64, device=DEV) % v.numel()
    return v[at].view(rows, 64)


def near(got, want, rel):
    bad = ~((got.double() - want).abs() <= (HALF + rel) * want.abs() + 1e-38)
    assert not bad.any(), (int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


# up to 16 rows; small tiles; one row of tiles with the sum in parts below; large tiles
@pytest.mark.parametrize("rows", [9, 100, 20000])
@pytest.mark.parametrize("lo,hi", [(-12.0, -8.0), (-8.0, -3.0), (-3.0, -0.25), (0.25, 20.0)])
def test_values(rows, lo, hi):
    z = grid(points(lo, hi), rows)
    one = torch.eye(64, dtype=torch.bfloat16, device=DEV)
    y, pre = mxq.moe_linear(z, one, activation="gelu", save_pre=True)
    assert torch.equal(pre, z)
    near(y, value(z.double()), TAIL)


def test_values_of_sums_in_parts():
    z = grid(points(-8.0, -3.0), 100)
    x = torch.zeros(100, 2048, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(64, 2048, dtype=torch.bfloat16, device=DEV)
    x[:, 960:1024], w[:, 960:1024] = z, torch.eye(64, dtype=torch.bfloat16, device=DEV)
    near(mxq.moe_linear(x, w, activation="gelu"), value(z.double()), TAIL)


@pytest.mark.parametrize("tokens", [1, 6, 40])
def test_the_layers_values(tokens):
    z = grid(points(-8.0, -3.0)[::3], tokens)
    one = torch.eye(64, dtype=torch.bfloat16, device=DEV)[None]
    y = mxq.moe_layer(z, torch.zeros(tokens, 1, device=DEV), one, one, 1, activation="gelu", gated=False)
    near(y, value(z.double()), TAIL + 2.0 ** -15)  # h in two bf16 parts


def test_slopes():
    """The gradient, whose two terms have opposite signs and differ by a factor
    of x^2 + 1: their errors count 1 + 2 / x^2 times at most, from -3 on down."""
    z = grid(points(-12.0, -3.0), 100)
    one = torch.eye(64, dtype=torch.bfloat16, device=DEV)
    dy = torch.ones_like(z)
    dx, _, db = mxq.moe_linear_backward(dy, z, one, pre=z, activation="gelu", bias=True)
    near(dx, slope(z.double()), 1.3 * TAIL)  # dz = dx: rounded once, multiplied by one
    want = slope(z.double())
    assert ((db[0].double() - want.sum(0)).abs() <= (1.3 * TAIL + 2.0 ** -18) * want.abs().sum(0)).all()


def test_infinities():
    z = torch.full((20, 64), float("-inf"), dtype=torch.bfloat16, device=DEV)
    z[:, ::2] = float("inf")
    one = torch.ones(64, 1, dtype=torch.bfloat16, device=DEV)
    y = mxq.moe_linear(z[:, :1], one, activation="gelu")
    assert (y == float("inf")).all()
    y = mxq.moe_linear(torch.full((20, 1), 1e38, dtype=torch.bfloat16, device=DEV), -one, activation="gelu")
    assert (y == 0).all()

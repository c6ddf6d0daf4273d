"""MXFP8 products and layers with e8m0 codes at the ends of their range, and what
an infinite weight reaches."""
import math

import pytest
import torch

import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ones(*shape):
    return torch.full(shape, 0x38, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)


def codes(code, *shape):
    return torch.full(shape, code, dtype=torch.uint8, device=DEV)


# up to 16 rows, small tiles, large tiles; scales in whole words and not
@pytest.mark.parametrize("rows,wide,width", [(3, 64, 128), (40, 64, 128), (40, 64, 160), (4096, 4096, 128), (4096, 4096, 160)])
def test_products(rows, wide, width):
    run = lambda xs, ws: mxq.moe_linear_mx(ones(rows, width), xs, ones(1, wide, width), ws)  # noqa: E731
    for code in (0, 1, 127, 253, 254):
        y = run(codes(254 - code, rows, width // 32), codes(code, 1, wide, width // 32))
        assert (y == width).all(), code
    # 255: NaN for the row, or the column, that has it, whichever its block
    for at in range(width // 32):
        xs, ws = codes(127, rows, width // 32), codes(127, 1, wide, width // 32)
        xs[rows - 1, at] = 255
        ws[0, 5, at] = 255
        y = run(xs, ws)
        assert y[rows - 1].isnan().all() and y[:, 5].isnan().all()
        keep = torch.arange(wide, device=DEV) != 5
        assert (y[:rows - 1, keep] == width).all()


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_layers(tokens):
    """Values that bf16 holds enter exactly, from e8m0 code 3 (its smallest value
    2^-133) to 246; 255 is NaN, for its expert's tokens alone."""
    one, logits = codes(127, 2, 64, 2), torch.zeros(tokens, 2, device=DEV)
    logits[:, 1] = 1.0
    new = lambda v: torch.full((tokens, 64), v, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    layer = lambda x, us, ds, uq=ones(2, 64, 64): mxq.moe_layer(  # noqa: E731
        x, logits, (uq, us), (ones(2, 64, 64), ds), 1, activation="none", gated=False)
    for code, scale in ((3, 2.0 ** 118), (60, 1.0), (246, 2.0 ** -125)):
        value = 2.0 ** (code - 127) * scale
        assert (layer(new(scale), codes(code, 2, 64, 2), one) == 4096 * value).all(), code
        assert (layer(new(scale / 64), one, codes(code, 2, 64, 2)) == 64 * value).all(), code
    # the smallest of the e4m3 values, 2^-9, times 2^(3 - 127)
    tiny = torch.full((2, 64, 64), 1, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    assert (layer(new(2.0 ** 120), codes(3, 2, 64, 2), one, tiny) == 4096 * 2.0 ** (120 - 133)).all()
    for which in ("up", "down"):
        bad = one.clone()
        bad[1, 7, 1] = 255
        other = one.clone()
        other[0, 7, 1] = 255  # of an expert that nobody takes
        y = layer(new(1.0), *((bad, one) if which == "up" else (one, bad)))
        assert y[:, 7].isnan().all() and (which == "up" or (y[:, :7] == 4096).all() and (y[:, 8:] == 4096).all())
        assert (layer(new(1.0), *((other, one) if which == "up" else (one, other))) == 4096).all()


@pytest.mark.parametrize("tokens", [3, 33])
def test_an_infinite_down_weight_stays_in_its_column(tokens):
    """h passes in two parts, so it comes out as NaN; for its expert's tokens alone."""
    up, down = (torch.ones(2, 64, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    down[1, 9, 3] = math.inf
    logits = torch.zeros(tokens, 2, device=DEV)
    logits[1, 1] = 1.0
    y = mxq.moe_layer(torch.ones(tokens, 64, dtype=torch.bfloat16, device=DEV), logits, up, down, 1, activation="none", gated=False)
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1, 9] = False
    assert (y[keep] == 4096).all() and not y[1, 9].isfinite()

"""Dense weights of 2 GiB and more, in memory or from the first row to the last:
every kernel takes them; of a gated product alone the reach is bounded."""
import pytest
import torch

import linear_reference as ref
import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = 2.0 ** -8
SUM = 2.0 ** -23


def normal(*shape, scale=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_().mul_(scale)


def near(got, want, size, terms):
    bad = ~((got.double() - want).abs() <= HALF * want.abs() + terms * size + 1e-30)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def ends_near(y, x, w, terms):
    """The first and the last columns against 64 bits, the rest by its size."""
    for at in (slice(0, 200), slice(-200, None)):
        m = w[at].double()
        near(y[:, at], x.double() @ m.t(), x.double().abs() @ m.abs().t(), terms)
    assert y.isfinite().all() and (y != 0).any(0).all()


@pytest.mark.parametrize("rows", [3, 17, 300])
def test_dense_weights(rows):
    torch.manual_seed(rows)
    w, x = normal(65536, 16384, scale=2.0 ** -7), normal(rows, 16384)
    ends_near(mxq.moe_linear(x, w), x, w, (16384 + 8) * SUM)


@pytest.mark.parametrize("rows,width", [(17, 64), (300, 64), (17, 63)])
def test_rows_far_apart(rows, width):
    """1100 rows, 2 MiB from one to the next; an odd length is copied together."""
    torch.manual_seed(rows)
    w = torch.empty(1100 << 20, dtype=torch.bfloat16, device=DEV).view(1100, 1 << 20)[:, :width]
    w.normal_().mul_(0.125)
    x = normal(rows, width)
    ends_near(mxq.moe_linear(x, w), x, w, (width + 8) * SUM)


@pytest.mark.parametrize("rows", [3, 17, 300])
def test_mx_rows_far_apart(rows):
    torch.manual_seed(rows)
    width, far = 128, 1 << 20
    w, x = normal(2100, width, scale=0.125), normal(rows, width)
    (wq, ws), (xq, xs) = mxq.quantize_mx_rowwise(w), mxq.quantize_mx_rowwise(x)
    big = torch.empty(2100 * far, dtype=torch.uint8, device=DEV).view(2100, far)[:, :width]
    big.copy_(wq.view(torch.uint8))
    y = mxq.moe_linear_mx(xq, xs, big.view(torch.float8_e4m3fn), ws)
    assert torch.equal(y, mxq.moe_linear_mx(xq, xs, wq, ws))


def test_gated_weights_are_refused():
    w = torch.empty(2048 << 20, dtype=torch.bfloat16, device=DEV).view(2048, 1 << 20)[:, :64]
    with pytest.raises(mxq.MXQError):
        mxq.moe_linear(normal(17, 64), w, gated=True)


def test_gated_rows_that_repeat():
    """One row for all 65536: little memory, whatever the rows' length."""
    torch.manual_seed(5)
    wide, width = 65536, 32768
    w, x = normal(1, width, scale=2.0 ** -7), normal(17, width)
    (wq, ws), (xq, xs) = mxq.quantize_mx_rowwise(w), mxq.quantize_mx_rowwise(x)
    y = mxq.moe_linear_mx(xq, xs, wq.view(torch.uint8).expand(wide, width).view(torch.float8_e4m3fn), ws.expand(wide, width // 32),
                          gated=True)
    assert torch.equal(y, y[:, :1].expand_as(y))
    a, b = ref.mx_values(xq, xs), ref.mx_values(wq, ws)[0]
    z, size = a @ b, a.abs() @ b.abs()
    # what the scaled instruction cuts, 2^-9 of the magnitudes, and the sum's additions; squared by the gate
    off = (2.0 ** -9 + (width + 8) * SUM) * size
    assert ((y[:, 0].double() - z * z).abs() <= HALF * z * z + (1 + HALF) * (2 * z.abs() * off + off * off)).all()

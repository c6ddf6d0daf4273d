"""Products of one row, whose stride says nothing: a row of an expanded tensor
(stride 0) or of overlapping ones (a stride shorter than the row) gives what its
contiguous copy gives."""
import pytest
import torch

import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def values(n, seed):
    return torch.randn(n, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def one_row(n, stride, seed):
    """(1, n) of that row stride, the memory behind it finite."""
    return values(n + 64 * max(stride, n), seed).as_strided((1, n), (stride, 1))


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


# small, medium and large tiles for the weight gradient; odd lengths are copied
@pytest.mark.parametrize("wide,width", [(8, 16), (64, 64), (40, 200), (2048, 1600), (4096, 4096), (33, 65)])
@pytest.mark.parametrize("stride", [0, 8, 1])
def test_gradients_of_one_row(wide, width, stride):
    dy, x, w = one_row(wide, stride, 1), one_row(width, stride, 2), values(wide * width, 3).view(1, wide, width)
    want = mxq.moe_linear_backward(dy.contiguous().clone(), x.contiguous().clone(), w, bias=True)
    assert same(mxq.moe_linear_backward(dy, x, w, bias=True), want)
    exact = dy[0].double()[:, None] * x[0].double()
    assert ((want[1][0].double() - exact).abs() <= 2.0 ** -8 * exact.abs()).all()  # one product each, one rounding
    # with a saved row and the gate's halves
    pre = one_row(wide * 2, stride, 4)
    w2 = values(2 * wide * width, 5).view(1, 2 * wide, width)
    kw = dict(activation="silu", gated=True, bias=True)
    want = mxq.moe_linear_backward(dy.contiguous().clone(), x.contiguous().clone(), w2, pre=pre.contiguous().clone(), **kw)
    assert same(mxq.moe_linear_backward(dy, x, w2, pre=pre, **kw), want)


@pytest.mark.parametrize("other", ["dy", "x"])
def test_an_infinity_beside_one_expanded_row(other):
    """One operand of stride 0, with an infinity: it reaches its row or column alone."""
    dy, x, w = values(64, 1).view(1, 64).clone(), values(64, 2).view(1, 64).clone(), values(64 * 64, 3).view(1, 64, 64)
    rows = {"dy": dy, "x": x}
    rows[other][0, 5] = float("inf")
    want = mxq.moe_linear_backward(dy, x, w)
    rows[other] = rows[other][0].expand(4, 64)[:1]
    got = mxq.moe_linear_backward(rows["dy"], rows["x"], w, need_x=False)
    assert torch.equal(got[1], want[1]) and not want[1].isnan().any()


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_one_row_of_weights(rows):
    """Experts of one row: what follows it in memory or repeats it takes no part."""
    width = 64
    w = values(width, 1)
    w[3] = float("inf")
    w = w.expand(4, width)[:1]
    dy, x = values(rows, 2).view(rows, 1), values(rows * width, 3).view(rows, width)
    got, want = mxq.moe_linear_backward(dy, x, w), mxq.moe_linear_backward(dy, x, w.contiguous().clone())
    assert same(got[:2], want[:2]) and not want[0].isnan().any()
    w = one_row(width, 0, 4)
    assert torch.equal(mxq.moe_linear(x, w), mxq.moe_linear(x, w.contiguous().clone()))
    assert torch.equal(mxq.moe_linear(x[0].expand(4, width)[:1], w), mxq.moe_linear(x[:1], w))

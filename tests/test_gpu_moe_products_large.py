"""The experts' products past 2^31 elements: long batches, wide results, many
large experts; and the layer's largest lists."""
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


def near(got, want, size, terms, what):
    bad = (got.double() - want).abs() > HALF * want.abs() + terms * SUM * size + 1e-30
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


def ends(*sizes):
    return torch.tensor(sizes).cumsum(0).to(torch.int32).to(DEV)


@pytest.mark.parametrize("width", [4096, 4095])
def test_long_batches(width):
    """The last groups of a batch of 2.2e9 elements, in place and copied."""
    torch.manual_seed(width)
    rows, wide, tail = 530000, 32, 77
    x, w = normal(rows, width), normal(3, wide, width, scale=width ** -0.5)
    offs = ends(rows - tail - 50, 50, tail - 9)
    y = mxq.moe_linear(x, w, offs)
    lo, hi = rows - tail, rows - 9
    want, size = x[lo:hi].double() @ w[2].double().t(), x[lo:hi].double().abs() @ w[2].double().abs().t()
    near(y[lo:hi], want, size, width + 8, "y")
    assert not y[hi:].any()
    dy = normal(rows, wide)
    dx, dw, db = mxq.moe_linear_backward(dy, x, w, offs, bias=True)
    d = dy[lo:hi].double()
    near(dx[lo:hi], d @ w[2].double(), d.abs() @ w[2].double().abs(), wide + 8, "dx")
    assert not dx[hi:].any()
    near(dw[2], d.t() @ x[lo:hi].double(), d.abs().t() @ x[lo:hi].double().abs(), tail + 8, "dw")
    torch.testing.assert_close(db[2].double(), d.sum(0), rtol=1e-5, atol=1e-4)


def test_wide_results():
    torch.manual_seed(1)
    rows, wide, width = 280000, 8192, 32
    x, w = normal(rows, width), normal(1, wide, width, scale=width ** -0.5)
    y, pre = mxq.moe_linear(x, w, activation="relu", save_pre=True)
    want, z, size = ref.forward(x[-300:].double(), w.double(), None, None, "relu")
    near(y[-300:], want, size, width + 8, "y")
    near(pre[-300:], z, size, width + 8, "z")
    dx, _, _ = mxq.moe_linear_backward(y, x, w, pre=pre, activation="relu", need_w=False)
    d = torch.where(pre[-300:] > 0, y[-300:], 0.0).double()
    near(dx[-300:], d @ w[0].double(), d.abs() @ w[0].double().abs(), wide + 8, "dx")


@pytest.mark.parametrize("per,width", [(4, 4096), (70, 4096), (4, 4095)])
def test_many_large_experts(per, width):
    """The last experts of 2.2e9 weights and of their gradient; few rows in all;
    MXFP8."""
    torch.manual_seed(per)
    E, wide = 530, 1024
    rows = E * per
    x, w = normal(rows, width), normal(E, wide, width, scale=width ** -0.5)
    offs = ends(*[per] * E)
    y = mxq.moe_linear(x, w, offs)
    last = x[-per:].double()
    want, size = last @ w[-1].double().t(), last.abs() @ w[-1].double().abs().t()
    near(y[-per:], want, size, width + 8, "y")
    dx, dw, _ = mxq.moe_linear_backward(y, x, w, offs)
    d = y[-per:].double()
    near(dx[-per:], d @ w[-1].double(), d.abs() @ w[-1].double().abs(), wide + 8, "dx")
    near(dw[-1], d.t() @ last, d.abs().t() @ last.abs(), per + 8, "dw")
    few = torch.zeros(E, dtype=torch.int32, device=DEV)
    few[-1] = per
    if per <= 16:
        near(mxq.moe_linear(x[-per:], w, few), want, size, width + 8, "few rows")
    del y, dx, dw
    if width % 32 == 0:
        wq, ws = mxq.quantize_mx_rowwise(w.view(-1, width))
        xq, xs = mxq.quantize_mx_rowwise(x)
        a, b = ref.mx_values(xq[-per:], xs[-per:]), ref.mx_values(wq[-wide:], ws[-wide:])
        want, size = a @ b.t(), a.abs() @ b.abs().t()
        wq, ws = wq.view(E, wide, width), ws.view(E, wide, -1)
        # 2^-9 of the magnitudes: what the scaled instruction cuts
        near(mxq.moe_linear_mx(xq, xs, wq, ws, offs)[-per:], want, size, 2 ** 14, "mx")
        if per <= 16:
            near(mxq.moe_linear_mx(xq[-per:], xs[-per:], wq, ws, few), want, size, 2 ** 14, "mx, few rows")


def test_the_layers_largest_weights():
    """Tokens that take the last of 4.3e9 up and 2.1e9 down weights."""
    torch.manual_seed(3)
    E, D, H = 520, 4096, 1024
    up, down = normal(E, 2 * H, D, scale=D ** -0.5), normal(E, D, H, scale=H ** -0.5)
    for T in (1, 5, 40):
        x, logits = normal(T, D), torch.full((T, E), -1e4, device=DEV)
        logits[:, -1] = 1.0
        y = mxq.moe_layer(x, logits, up, down, 1)
        h, _, size = ref.forward(x.double(), up[-1:].double(), None, None, "silu", True)
        want = h @ down[-1].double().t()
        # sums over D, h in 16 bits, sums over H
        bound = ((D + 8) * SUM * size + 2e-5 * h.abs() + (H + 40) * SUM * h.abs()) @ down[-1].double().abs().t()
        assert ((y.double() - want).abs() <= HALF * want.abs() + 1.01 * bound).all(), T


def test_the_layers_longest_lists():
    """64 tokens, 32 slots each, over 1024 experts: as the operators one by one."""
    torch.manual_seed(4)
    T, E, k, D, H = 64, 1024, 32, 64, 32
    x, logits = normal(T, D), torch.randn(T, E, device=DEV)
    up, down = normal(E, 2 * H, D, scale=D ** -0.5), normal(E, D, H, scale=H ** -0.5)
    y = mxq.moe_layer(x, logits, up, down, k)
    r = mxq.moe_route(logits, k, align=1)
    h = mxq.moe_linear(mxq.moe_dispatch(x, r), up, r.offs, activation="silu", gated=True)
    chain = mxq.moe_combine(mxq.moe_linear(h, down, r.offs), r)
    # there h and the experts' results are rounded to bf16 too
    assert torch.linalg.vector_norm(y.double() - chain.double()) < 2 * HALF * torch.linalg.vector_norm(chain.double())


def test_one_token_masked_or_barred():
    x, logits = normal(1, 64), torch.randn(1, 8, device=DEV)
    up, down = normal(8, 64, 64), normal(8, 64, 32)
    off = torch.zeros(1, dtype=torch.bool, device=DEV)
    assert not mxq.moe_layer(x, logits, up, down, 3, token_mask=off).any()
    assert torch.equal(mxq.moe_layer(x, logits, up, down, 3, token_mask=off, residual=x), x)
    barred = torch.full_like(logits, float("-inf"))
    assert not mxq.moe_layer(x, barred, up, down, 3).any()
    barred[0, 5] = -1e30
    one = mxq.moe_layer(x, barred, up, down, 3)
    logits[0, 5] = 1e30
    assert torch.equal(one, mxq.moe_layer(x, logits, up, down, 1)) and one.any()

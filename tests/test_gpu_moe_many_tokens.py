"""Token counts past what one launch's grid takes (2^26 pieces of work, 2^24
tokens for the wide combine gradient): every token is reached, padding rows
are cleared once and for all."""
import pytest
import torch

import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def route(T, rows, align=1, offs=None):
    i32 = dict(dtype=torch.int32, device=DEV)
    return mxq.MoeRoute(weights=torch.full((T, 1), 2.0, device=DEV), rows=rows, counts=torch.tensor([T], **i32),
                        offs=torch.tensor([T if offs is None else offs], **i32), align=align)


def test_narrow_rows():
    T, W = (1 << 26) + 77, 2
    rows = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV).reshape(T, 1)
    r = route(T, rows, align=6, offs=(T + 5) // 6 * 6)
    x = torch.arange(T * W, dtype=torch.int32, device=DEV).remainder_(251).sub_(125).to(torch.bfloat16).reshape(T, W)
    cap = mxq.moe_row_capacity(T, 1, 1, 6)
    xg = mxq.moe_dispatch(x, r)
    assert xg.shape == (cap, W) and cap == T + 5
    assert torch.equal(xg[:T], x.flip(0)) and not xg[T:].any()
    assert torch.equal(mxq.moe_combine(xg, r, residual=x), x * 3)
    assert torch.equal(mxq.moe_dispatch_backward(xg, r), x)
    dyg, dw = mxq.moe_combine_backward(x, xg, r)
    assert torch.equal(dyg[:T], xg[:T] * 2) and not dyg[T:].any()
    assert torch.equal(dw[:, 0], x.float().square_().sum(1))


@pytest.mark.parametrize("T,W", [((1 << 25) + 9, 4096), ((1 << 24) + 50, 1032)])
def test_wide_rows_few_of_them_taken(T, W):
    """A row that repeats; of the tokens only some have a slot, past the end
    of the first launch among them."""
    at = torch.tensor([0, 5, T // 2, T // 2 + 1, T - 40, T - 2, T - 1], device=DEV)
    rows = torch.full((T, 1), -1, dtype=torch.int32, device=DEV)
    rows[at, 0] = torch.arange(len(at), dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    n = len(at)
    w = torch.rand(T, 1, device=DEV)
    r = mxq.MoeRoute(weights=w, rows=rows, counts=torch.tensor([n], **i32), offs=torch.tensor([n], **i32))
    x = (torch.arange(W, device=DEV).remainder(17) - 8).to(torch.bfloat16)
    out = torch.full((n + 2, W), 7.0, dtype=torch.bfloat16, device=DEV)
    code = mxq.mxq_moe_dispatch(x.data_ptr(), mxq.MXQ_BF16, T, W, 0, 1, rows.data_ptr(), 1, r.counts.data_ptr(),
                                r.offs.data_ptr(), 1, out.data_ptr(), n + 2, W, 1,
                                torch.cuda.current_stream().cuda_stream)
    assert code == 0
    assert torch.equal(out[:n], x.expand(n, W)) and not out[n:].any()
    dyg, dw = mxq.moe_combine_backward(x.expand(T, W), out, r)
    assert torch.equal(dyg[:n], (w[at] * x.float()).to(torch.bfloat16)) and not dyg[n:].any()
    want = torch.zeros(T, device=DEV)
    want[at] = float(x.double().square().sum())  # a whole number below 2^24: exact in fp32
    assert torch.equal(dw[:, 0], want)


def test_the_most_tokens_that_a_route_takes():
    """2^31 - 1 tokens: the last run's end and the step past its last round
    are past 31 bits."""
    T = (1 << 31) - 1
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    mask[7] = mask[T - 3] = False
    r = mxq.moe_route(torch.zeros((T, 1), dtype=torch.bfloat16, device=DEV), 1, token_mask=mask)
    del mask
    assert int(r.live) == T - 2 and r.counts.tolist() == [T - 2] and r.offs.tolist() == [T - 2]
    assert r.mean_prob.tolist() == [1.0] and r.losses.tolist() == [1.0, 0.0]
    want = torch.arange(T, dtype=torch.int32, device=DEV)
    want[8:] -= 1
    want[T - 2:] -= 1
    want[7] = want[T - 3] = -1
    assert torch.equal(r.rows[:, 0], want)
    assert torch.equal(r.ids[:, 0], want.clamp_(-1, 0))
    assert torch.equal(r.weights[:, 0], want.add_(1).float())
    assert not r.lse[:7].any() and torch.isinf(r.lse[[7, T - 3]]).all() and not r.lse[T - 2:].any()

"""Group ends that decrease, which the products' contract leaves open: the bias
gradient's sums stay in their part of the workspace, and its neighbours' bytes as
they were.  Ends that keep the contract give what they gave."""
import pytest
import torch

import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def bias_gradient(dy, offs, pre, act, gated, wide, behind):
    """grad_bias alone, the workspace followed by `behind` bytes of 0xa5."""
    rows, E = dy.shape[0], offs.numel()
    none = mxq.ACTIVATIONS[act]
    saved = act != "none" or gated
    need = mxq.mxq_moe_linear_backward_workspace_bytes(rows, 8, E, wide, none, int(gated), 1, 1)
    buf = torch.full((need + behind,), 0xa5, dtype=torch.uint8, device=DEV)
    out = torch.full((E + 2, wide), -7.0, device=DEV)
    code = mxq.mxq_moe_linear_backward(
        dy.data_ptr(), dy.stride(0), 1, 0, rows, 8, 8, 1, 0, E, wide, wide * 8, 8, 1, offs.data_ptr(),
        pre.data_ptr() if saved else 0, wide, 1, none, int(gated), 0, 8, 1, 0, wide * 8, 8, 1, out[1].data_ptr(),
        buf.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    torch.cuda.synchronize()
    assert (out[0] == -7).all() and (out[-1] == -7).all()
    return out[1:-1], buf[need:]


# slices of 16 and of 64 rows
@pytest.mark.parametrize("rows,E,n", [(1000, 64, 64), (8192, 64, 4096), (300, 1000, 40)])
@pytest.mark.parametrize("act,gated", [("none", False), ("relu", False), ("silu", True)])
def test_the_sums_stay_in_their_space(rows, E, n, act, gated):
    wide = 2 * n if gated else n
    torch.manual_seed(rows)
    dy = torch.randn(rows, n, device=DEV).to(torch.bfloat16)
    pre = torch.randn(rows, wide, device=DEV).to(torch.bfloat16)
    behind = 1 << 22
    for offs in ([rows, 0] * (E // 2), list(range(rows, 0, -max(rows // E, 1)))[:E] + [0] * max(E - rows, 0)):
        offs = torch.tensor((offs + [0] * E)[:E], dtype=torch.int32, device=DEV)
        _, rest = bias_gradient(dy, offs, pre, act, gated, wide, behind)
        assert (rest == 0xa5).all()
    # sorted ends: the sums of each group
    offs = torch.randint(0, rows + 1, (E,), device=DEV).sort().values.to(torch.int32)
    got, rest = bias_gradient(dy, offs, pre, act, gated, wide, behind)
    assert (rest == 0xa5).all()
    if act == "none":
        upto = torch.cat([torch.zeros(1, n, dtype=torch.float64, device=DEV), dy.double().cumsum(0)])
        ends = torch.cat([offs.new_zeros(1), offs]).long()
        want = upto[ends[1:]] - upto[ends[:-1]]
        size = torch.cat([torch.zeros(1, n, dtype=torch.float64, device=DEV), dy.double().abs().cumsum(0)])
        size = size[ends[1:]] - size[ends[:-1]]
        # sums of up to 64 values in fp32, of those in fp64, one rounding
        assert ((got.double() - want).abs() <= 2.0 ** -18 * size + 1e-12).all()

"""Checks of the tensor-level routing calls that need no GPU."""
import pytest
import torch

import mxfp8_quantization_moe_amd as mxq
from mxfp8_quantization_moe_amd import moe


class OnDevice(torch.Tensor):
    """A host tensor that says it is on the GPU, for checks made before a launch."""
    is_cuda = property(lambda self: True)


def route(T, k, E, **kw):
    i32 = dict(dtype=torch.int32)
    r = mxq.MoeRoute(weights=torch.ones(T, k), rows=torch.zeros(T, k, **i32), counts=torch.zeros(E, **i32),
                     offs=torch.zeros(E, **i32))
    return r._replace(**kw)


@pytest.mark.parametrize("weights", [None, torch.ones(9, 2), torch.ones(10, 1), torch.ones(10, 2, dtype=torch.float64),
                                     torch.ones(2, 10).t()])
def test_combine_needs_the_routes_weights(weights, monkeypatch):
    """Without weights the C call adds the rows up as they are, which is the
    dispatch's gradient and not a combine."""
    monkeypatch.setattr(moe, "_run", lambda t, stream, call: "launched")
    yg = torch.zeros(20, 16).as_subclass(OnDevice)
    assert mxq.moe_combine(yg, route(10, 2, 4)) == "launched"
    with pytest.raises(TypeError, match="route.weights"):
        mxq.moe_combine(yg, route(10, 2, 4, weights=weights))
    assert mxq.moe_dispatch_backward(yg, route(10, 2, 4, weights=weights)) == "launched"

"""Refusals of the products' binding that need no GPU."""
import pytest
import torch

import mxfp8_quantization_moe_amd as mxq


def test_refusals_without_a_gpu():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 6, 8, dtype=torch.bfloat16)
    offs = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mxq.moe_linear(x, w, offs), lambda: mxq.moe_linear_backward(x, x, w, offs),
                 lambda: mxq.moe_linear_mx(x, offs, w, offs, offs)):
        with pytest.raises(TypeError):
            call()
    assert set(mxq.ACTIVATIONS) == {"none", "relu", "gelu", "silu"}
    assert [mxq.ACTIVATIONS[n] for n in ("none", "relu", "gelu", "silu")] == [0, 1, 2, 3]

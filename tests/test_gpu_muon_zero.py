"""A matrix of zeros stays zeros whatever eps is, and leaves the others of its
call alone."""
import pytest
import torch

import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-7, 1e-3])
@pytest.mark.parametrize("steps", [0, 1, 5])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_zero_matrix_gives_zeros(eps, steps, dtype):
    g = torch.randn(3, 70, 90, generator=torch.Generator().manual_seed(1)).to(dtype).to("cuda:0")
    g[1] = 0
    out = mxq.muon_orthogonalize(g, eps=eps, steps=steps)
    assert (out[1] == 0).all()
    both = mxq.muon_orthogonalize(g[[0, 2]], eps=eps, steps=steps)
    assert torch.isfinite(both).all() and torch.equal(out[[0, 2]], both)

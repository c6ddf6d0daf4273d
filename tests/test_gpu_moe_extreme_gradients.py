"""The router's gradient for logits far from zero: rows barred altogether with
a finite value, offsets common to a row, the ends of the number range."""
import numpy as np
import pytest
import torch

import moe_exact as ref
import mxfp8_quantization_moe_amd as mxq
from test_gpu_moe_extremes import RTOL, SIZES, logits

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(l, k, renorm, dtype, gl):
    """The softmax' Jacobian and the z loss' gradient, each within RTOL (fp32,
    see test_gpu_moe_extremes) of the magnitudes that it adds up."""
    T, E = l.shape
    want = ref.route(l.double().numpy(), k, None, renorm)
    r = mxq.moe_route(l.to(DEV), k, renormalize=renorm)
    gw = np.random.default_rng(7).normal(size=(T, k)).astype(np.float32)
    gl = np.array(gl, np.float32)
    n = max(want["live"], 1)
    for use_w in (True, False):
        d = mxq.moe_route_backward(l.to(DEV), r, torch.from_numpy(gw).to(DEV) if use_w else None,
                                   torch.from_numpy(gl).to(DEV)).double().cpu().numpy()
        w = ref.route_backward(want, k, renorm, gw.astype(np.float64) if use_w else None, gl.astype(np.float64))
        size = np.full((T, 1), gl[0] * E * want["counts"].max() / (n * n * k) * 2)
        if use_w:
            sel = np.where(want["ids"] >= 0, np.take_along_axis(want["p"], np.maximum(want["ids"], 0), 1), 0).sum(1)
            size += (np.abs(gw).max(1) / np.where(renorm & (sel > 0), sel, 1.0))[:, None] * 4
        size += (gl[1] * 2 / n * np.abs(np.where(np.isfinite(want["lse"]), want["lse"], 0)))[:, None]
        tol = RTOL * want["p"] * size + 1e-30
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(w)  # rounded to 8 significant bits
        bad = ~(np.abs(d - w) <= tol)
        assert not bad.any(), (use_w, renorm, np.argwhere(bad)[:5].tolist(), d[bad][:5], w[bad][:5])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_extreme_rows(T, E, k, dtype):
    l, _ = logits(T, E, dtype, T + E)
    for renorm in (True, False):
        check(l, k, renorm, dtype, (0.5, 0.0))
        check(l, k, renorm, dtype, (0.5, 0.25))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [1e3, -1e4, 3e5, -1e9])
def test_offsets_common_to_a_row(offset, dtype):
    g = torch.Generator().manual_seed(5)
    for T, E, k in ((50, 8, 2), (200, 61, 6), (90, 256, 8)):
        l = (1.5 * torch.randn(T, E, generator=g) + offset * torch.rand(T, 1, generator=g)).to(dtype)
        for renorm in (True, False):
            check(l, k, renorm, dtype, (0.5, 0.0))


def test_an_expert_that_is_not_available_has_no_gradient_beside_a_large_z_gradient():
    """p = 0 stays 0 where the z loss' factor 2 g lse / n passes fp32's range."""
    l = torch.zeros(1, 8)
    l[0] = torch.finfo(torch.float32).min
    l[0, 2:5] = -float("inf")
    r = mxq.moe_route(l.to(DEV), 2)
    d = mxq.moe_route_backward(l.to(DEV), r, None, torch.tensor([0.0, 0.75], device=DEV))[0].cpu()
    assert (d[2:5] == 0).all()
    # 2 * 0.75 * lse * p with p = 1 / 5
    np.testing.assert_allclose(d[[0, 1, 5, 6, 7]].double(), 1.5 * torch.finfo(torch.float32).min / 5, rtol=RTOL)

"""Training batches through the router's large-batch path (many runs of
tokens, each thread of the scan with several of them) against 64 bits."""
import numpy as np
import pytest
import torch

import moe_exact as ref
import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
RTOL = 1e-5  # fp32, derived in test_gpu_moe_route


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,align", [
    (16384, 256, 8, 16),    # 256 runs of one round
    (16390, 61, 6, 32),     # 129 runs of two rounds, the last of 6 tokens
    (20000, 256, 4, 1),     # 157 runs of two rounds
    (33333, 130, 9, 48),    # 174 runs of three rounds
    (6000, 700, 3, 16),     # 94 runs
    (5000, 2000, 12, 7),    # 79 runs, 64 experts per lane
])
def test_batches(T, E, k, align, dtype):
    g = torch.Generator().manual_seed(T + E)
    l = 1.5 * torch.randn(T, E, generator=g) + 0.5 * torch.randn(1, E, generator=g)
    off = torch.rand(T, (E + 7) // 8, generator=g) < 0.3
    l[off.repeat_interleave(8, 1)[:, :E]] = -float("inf")
    l[T // 3] = -float("inf")
    l = l.to(dtype)
    mask = torch.rand(T, generator=g) < 0.85
    want = ref.route(l.double().numpy(), k, mask.numpy(), True, align)
    dev = l.to(DEV)
    r = mxq.moe_route(dev, k, token_mask=mask.to(DEV), align=align)
    for name in ("ids", "counts", "offs", "rows"):
        assert np.array_equal(getattr(r, name).cpu().numpy(), want[name]), name
    assert int(r.live) == want["live"]
    for name in ("weights", "mean_prob", "losses"):
        np.testing.assert_allclose(getattr(r, name).double().cpu().numpy(), want[name], rtol=RTOL, atol=1e-30,
                                   err_msg=name)
    np.testing.assert_allclose(r.lse.double().cpu().numpy(), want["lse"], rtol=RTOL, atol=4e-6)

    gw = torch.randn(T, k, generator=g)
    gl = np.array([0.5, 0.25], np.float32)
    d = mxq.moe_route_backward(dev, r, gw.to(DEV), torch.from_numpy(gl).to(DEV)).double().cpu().numpy()
    w = ref.route_backward(want, k, True, gw.double().numpy(), gl.astype(np.float64))
    n = want["live"]
    sel = np.where(want["ids"] >= 0, np.take_along_axis(want["p"], np.maximum(want["ids"], 0), 1), 0).sum(1)
    size = (gw.abs().amax(1).numpy() / np.where(sel > 0, sel, 1.0))[:, None] * 4
    size = size + gl[0] * E * want["counts"].max() / (n * n * k) * 2
    size = size + (gl[1] * 2 / n * np.abs(np.where(np.isfinite(want["lse"]), want["lse"], 0)))[:, None]
    tol = RTOL * want["p"] * size + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(w)
    assert (np.abs(d - w) <= tol).all()

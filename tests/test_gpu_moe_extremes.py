"""Router rows at the ends of the number range beside ordinary ones: every
expert barred with the type's lowest value or another large finite one, the
largest value alone, large offsets; probabilities, statistics and losses
against 64 bits."""
import numpy as np
import pytest
import torch

import moe_exact as ref
import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# fp32: exp(x) for -24 <= x <= 0 is off by (1 + 1.5 * 24) 2^-24 = 2.2e-6 of
# itself at most (the rounding of x log2 e), a sum of E <= 1500 terms adds less
# than 1e-6, a quotient doubles both: below 1e-5.  Differences below -24 belong
# to probabilities under 4e-11, off by less than |x| * 2^-23 < 1e-5 of
# themselves down to 2^-126.
RTOL = 1e-5


def logits(T, E, dtype, seed):
    """Ordinary rows and, from row 1 on, one of each extreme kind."""
    g = torch.Generator().manual_seed(seed)
    l = 1.5 * torch.randn(T, E, generator=g)
    low, top = torch.finfo(dtype).min, torch.finfo(dtype).max
    l = l.to(dtype).float()
    kinds = [
        [low] * E,                                        # barred altogether with the lowest finite value
        [low] * (E - 1) + [1.5],                          # but for one
        [top] + [low] * (E - 1),
        [top] * E,
        [2.4e38] + [0.5] * (E - 1),
        [-2.4e38] * E,
        [-1e9] * E,                                       # another usual bar
        [-1e9] * (E // 2) + [0.25] * (E - E // 2),
        [-float("inf")] * (E // 2) + [low] * (E - E // 2),
        [1e30] * E,
        [-1e4] * E,
    ]
    for i, row in enumerate(kinds):
        l[1 + 2 * i] = torch.tensor(row)
    return l.to(dtype), 1 + 2 * np.arange(len(kinds))


SIZES = [(64, 8, 2), (30, 61, 6), (300, 8, 2), (200, 64, 8), (500, 256, 8), (130, 300, 20), (100, 1500, 4)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_probabilities_of_extreme_rows(T, E, k, dtype):
    l, _ = logits(T, E, dtype, T + E)
    for renorm in (True, False):
        want = ref.route(l.double().numpy(), k, None, renorm, 4)
        r = mxq.moe_route(l.to(DEV), k, renormalize=renorm, align=4)
        for name in ("ids", "counts", "offs", "rows"):
            assert np.array_equal(getattr(r, name).cpu().numpy(), want[name]), name
        assert int(r.live) == T
        for name in ("weights", "mean_prob"):
            np.testing.assert_allclose(getattr(r, name).double().cpu().numpy(), want[name], rtol=RTOL, atol=1e-30,
                                       err_msg=name)
        np.testing.assert_allclose(r.lse.double().cpu().numpy(), want["lse"], rtol=RTOL, atol=4e-6)
        np.testing.assert_allclose(float(r.losses[0]), want["losses"][0], rtol=RTOL)
        # the mean of lse^2 is past fp32 with these rows, whatever its sum is held in
        assert want["losses"][1] > 1e70 and float(r.losses[1]) == float("inf")


@pytest.mark.parametrize("E", [8, 256])
def test_losses_beside_rows_with_a_finite_bar(E):
    """Rows barred altogether with -1e4 or -1e9: both losses are finite."""
    g = torch.Generator().manual_seed(E)
    for T, bar in ((50, -1e4), (700, -1e9)):
        l = torch.randn(T, E, generator=g)
        l[7] = bar
        l[11, 1:] = bar
        want = ref.route(l.double().numpy(), 2)
        r = mxq.moe_route(l.to(DEV), 2)
        for name in ("weights", "mean_prob", "losses"):
            np.testing.assert_allclose(getattr(r, name).double().cpu().numpy(), want[name], rtol=RTOL, atol=1e-30,
                                       err_msg=name)

"""The whole-array 64-bit router against the one written token by token."""
import numpy as np
import pytest

import moe_exact
import moe_reference


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 3), (40, 4, 4), (30, 16, 2)])
def test_the_two_forms_agree(T, E, k, renorm):
    g = np.random.default_rng(T * 100 + E)
    l = (2 * g.normal(size=(T, E))).round(1)  # with ties
    mask = g.random(T) < 0.8
    if T > 4:
        l[2] = -np.inf
        l[3, : E - 1] = -np.inf
        mask[2:4] = True
    a, b = moe_exact.route(l, k, mask, renorm, 4), moe_reference.route(l, k, mask, renorm, 4)
    for name in ("ids", "rows", "counts", "offs", "live"):
        assert np.array_equal(a[name], b[name]), name
    for name in ("weights", "lse", "p", "mean_prob", "losses"):
        np.testing.assert_allclose(a[name], b[name], rtol=1e-12, atol=1e-14, err_msg=name)
    gl = np.array([0.7, 0.3])
    for gw in (None, g.normal(size=(T, k))):
        x, y = moe_exact.route_backward(a, k, renorm, gw, gl), moe_reference.route_backward(b, k, renorm, gw, gl)
        np.testing.assert_allclose(x, y, rtol=1e-12, atol=1e-14)

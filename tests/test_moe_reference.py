"""The tests' 64-bit router gradient against difference quotients of the
router's own objective (selection and counts held fixed)."""
import numpy as np
import pytest

import moe_reference as ref


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 3), (9, 4, 4), (6, 16, 2)])
def test_route_gradient_matches_differences(T, E, k, renorm):
    g = np.random.default_rng(T * 100 + E)
    l = g.normal(size=(T, E)) * 1.5
    mask = np.ones(T, bool)
    if T > 4:
        mask[1] = False
        l[2] = -np.inf
        l[3, : E - 1] = -np.inf
    r = ref.route(l, k, mask, renorm)
    gw, gl = g.normal(size=(T, k)), np.array([0.7, 0.3])
    d = ref.route_backward(r, k, renorm, gw, gl)
    n = max(r["live"], 1)
    # central differences with h = 1e-5: truncation h^2 * |f'''| / 6 ~ 1e-10,
    # rounding 2^-52 * |f| / h ~ 1e-10
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if l[t, e] == -np.inf:
                assert d[t, e] == 0
                continue
            up, dn = l.copy(), l.copy()
            up[t, e] += h
            dn[t, e] -= h
            f = [ref.route_objective(x, k, r["ids"], r["counts"], n, mask, renorm, gw, gl) for x in (up, dn)]
            assert abs((f[0] - f[1]) / (2 * h) - d[t, e]) < 1e-8

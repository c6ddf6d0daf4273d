"""Plain 64-bit forms of the mixture-of-experts operators for the tests,
written loop by loop or with numpy from the definitions in include/mxq.h."""
from __future__ import annotations

import numpy as np


def route(logits, k, mask=None, renorm=True, align=1):
    """logits: float64 (T, E)."""
    T, E = logits.shape
    ids = np.full((T, k), -1, np.int64)
    w = np.zeros((T, k))
    lse = np.full(T, np.inf)
    p = np.zeros((T, E))
    for t in range(T):
        l = logits[t]
        if (mask is not None and not mask[t]) or not (l > -np.inf).any():
            continue
        top = np.nanmax(l)
        with np.errstate(invalid="ignore"):
            lse[t] = np.log(np.exp(l - top).sum()) + top
            p[t] = np.exp(l - lse[t])
        order = sorted((e for e in range(E) if l[e] > -np.inf), key=lambda e: (-l[e], e))[:k]
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
        if renorm:
            w[t] /= p[t, order].sum()
    live = np.isnan(lse) | (lse < np.inf)
    n = int(live.sum())
    counts = np.array([(ids == e).sum() for e in range(E)])
    ends = np.cumsum((counts + align - 1) // align * align)
    starts = ends - (counts + align - 1) // align * align
    rows = np.full((T, k), -1, np.int64)
    used = np.zeros(E, np.int64)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e >= 0:
                rows[t, j] = starts[e] + used[e]
                used[e] += 1
    nf = max(n, 1)
    mean = p.sum(0) / nf
    losses = np.array([E * (counts / (nf * k) * mean).sum(), (lse[live] ** 2).sum() / nf])
    return dict(ids=ids, weights=w, lse=lse, p=p, counts=counts, offs=ends, rows=rows, mean_prob=mean, losses=losses,
                live=n)


def route_objective(logits, k, ids, counts, n, mask, renorm, gw, gl):
    """The scalar <gw, weights> + <gl, losses> with the selection and the
    counts held fixed, for difference quotients."""
    T, E = logits.shape
    total, mean, z = 0.0, np.zeros(E), 0.0
    for t in range(T):
        l = logits[t]
        if (mask is not None and not mask[t]) or not (l > -np.inf).any():
            continue
        lse = np.log(np.exp(l - l.max()).sum()) + l.max()
        p = np.exp(l - lse)
        sel = [e for e in ids[t] if e >= 0]
        w = p[sel] / (p[sel].sum() if renorm else 1.0)
        total += (gw[t, :len(sel)] * w).sum()
        mean += p
        z += lse * lse
    return total + gl[0] * E * (counts / (n * k) * mean / n).sum() + gl[1] * z / n


def route_backward(r, k, renorm, gw, gl):
    p, ids, counts, n = r["p"], r["ids"], r["counts"], max(r["live"], 1)
    T, E = p.shape
    d = np.zeros((T, E))
    for t in range(T):
        if r["lse"][t] == np.inf:
            continue
        g = gl[0] * E * counts / (n * k) / n
        sel = [e for e in ids[t] if e >= 0]
        if gw is not None:
            q = gw[t, :len(sel)].copy()
            if renorm:
                s = p[t, sel].sum()
                q = (q - (q * p[t, sel]).sum() / s) / s
            g = g.copy()
            g[sel] += q
        d[t] = p[t] * (g - (p[t] * g).sum()) + gl[1] * 2 * r["lse"][t] * p[t] / n
    return d


def dispatch(x, rows, cap):
    out = np.zeros((cap, x.shape[1]))
    for t, j in zip(*np.nonzero(rows >= 0)):
        out[rows[t, j]] = x[t]
    return out


def combine(yg, rows, w, residual=None):
    y = np.zeros((rows.shape[0], yg.shape[1])) if residual is None else residual.astype(np.float64).copy()
    for t, j in zip(*np.nonzero(rows >= 0)):
        y[t] += (1.0 if w is None else w[t, j]) * yg[rows[t, j]]
    return y


def combine_backward(dy, yg, rows, w):
    dyg, dw = np.zeros_like(yg), np.zeros(rows.shape)
    for t, j in zip(*np.nonzero(rows >= 0)):
        dyg[rows[t, j]] = w[t, j] * dy[t]
        dw[t, j] = (dy[t] * yg[rows[t, j]]).sum()
    return dyg, dw

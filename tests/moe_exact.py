"""The router's definitions in 64 bits over whole arrays: probabilities as
exponentials over their sum, so that rows of any finite size keep them (an
exponential of l - lse loses the sum beside a large lse), and fast enough for
batches of many thousand tokens."""
from __future__ import annotations

import numpy as np


def route(logits, k, mask=None, renorm=True, align=1):
    """logits: float64 (T, E) without NaN and +inf."""
    T, E = logits.shape
    live = (logits > -np.inf).any(1)
    if mask is not None:
        live &= mask
    n = int(live.sum())
    safe = np.where(live[:, None], logits, 0.0)
    top = safe.max(1, keepdims=True)
    ex = np.exp(safe - top)
    total = ex.sum(1, keepdims=True)
    p = np.where(live[:, None], ex / total, 0.0)
    lse = np.where(live, (np.log(total) + top)[:, 0], np.inf)
    ids = np.argsort(-safe, axis=1, kind="stable")[:, :k]
    taken = (np.take_along_axis(safe, ids, 1) > -np.inf) & live[:, None]
    w = np.where(taken, np.take_along_axis(p, ids, 1), 0.0)
    if renorm:
        w = w / np.where(live, w.sum(1), 1.0)[:, None]
    hit = np.zeros((T, E), np.int64)
    np.put_along_axis(hit, ids, taken.astype(np.int64), 1)
    counts = hit.sum(0)
    lengths = (counts + align - 1) // align * align
    offs = np.cumsum(lengths)
    at = (offs - lengths)[None, :] + np.cumsum(hit, 0) - hit
    nf = max(n, 1)
    mean = p.sum(0) / nf
    losses = np.array([E * (counts / (nf * k) * mean).sum(), np.square(lse[live]).sum() / nf])
    return dict(ids=np.where(taken, ids, -1), weights=w, lse=lse, p=p, counts=counts, offs=offs,
                rows=np.where(taken, np.take_along_axis(at, ids, 1), -1), mean_prob=mean, losses=losses, live=n)


def route_backward(r, k, renorm, gw, gl):
    """gw: (T, k) or None; gl: (balance, z)."""
    p, ids, n = r["p"], r["ids"], max(r["live"], 1)
    T, E = p.shape
    g = np.tile(gl[0] * E * r["counts"] / (n * k) / n, (T, 1))
    if gw is not None:
        taken, at = ids >= 0, np.maximum(ids, 0)
        q = np.where(taken, gw, 0.0)
        if renorm:
            s = np.where(taken, np.take_along_axis(p, at, 1), 0.0).sum(1, keepdims=True)
            q = np.where(taken, (q - (q * r["weights"]).sum(1, keepdims=True)) / np.where(s > 0, s, 1.0), 0.0)
        for j in range(k):  # an empty slot adds its 0 to expert 0
            g[np.arange(T), at[:, j]] += q[:, j]
    lse = np.where(np.isfinite(r["lse"]), r["lse"], 0.0)
    return p * (g - (p * g).sum(1, keepdims=True)) + gl[1] * 2 / n * lse[:, None] * p

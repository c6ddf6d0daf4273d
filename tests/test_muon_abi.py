"""Argument checks of the Newton-Schulz C entry points; no GPU is touched."""
import pytest

from mxfp8_quantization_moe_amd import _capi, build

A = 1 << 20  # a plausible, aligned address; every call here returns before a launch
NEED = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return _capi.load()


def test_workspace_bytes(lib):
    need = lib.mxq_muon_workspace_bytes
    for bad in ((-1, 4, 4), (1, -1, 4), (1, 4, -1), (1, 65537, 4), (1, 4, 65537), (65536, 4, 4)):
        assert need(*bad) == -1, bad
    assert need(0, 4, 4) == need(1, 0, 4) == need(1, 4, 0) == 0
    for m, n in ((1, 1), (64, 64), (100, 777), (2048, 768), (8192, 5120)):
        one, tall = need(1, m, n), need(1, n, m)
        assert one == tall
        # X in two parts twice (the f16 one), A in two, B in one
        lo, hi = min(m, n), max(m, n)
        assert one >= 5 * lo * hi + 5 * lo * lo
        assert need(3, m, n) >= 3 * (5 * lo * hi + 5 * lo * lo)


def test_refusals(lib):
    d = dict(g=A, dt=0, count=2, rows=64, cols=96, ge=64 * 96, gr=96, gc=1, out=A, oe=64 * 96, orr=96, oc=1, steps=5,
             a=3.0, b=-4.0, c=2.0, eps=1e-7, scale=1.0, ws=A, bytes=NEED)

    def call(**kw):
        return lib.mxq_muon_orthogonalize(*dict(d, **kw).values(), None)

    for kw in (dict(g=0), dict(out=0), dict(dt=2), dict(dt=-1), dict(count=-1), dict(rows=-1), dict(cols=65537),
               dict(count=65536), dict(steps=-1), dict(steps=1001), dict(eps=-1.0), dict(eps=float("nan")),
               dict(g=A + 1), dict(dt=1, g=A + 2), dict(out=A + 1), dict(ws=A + 8)):
        assert call(**kw) == 1, kw
    for kw in (dict(gc=2), dict(oc=2), dict(gr=2, gc=3)):
        assert call(**kw) == 2, kw
    short = lib.mxq_muon_workspace_bytes(2, 64, 96) - 1
    for kw in (dict(bytes=short), dict(bytes=0), dict(ws=0)):
        assert call(**kw) == 4, kw
    for kw in (dict(count=0), dict(rows=0), dict(cols=0)):
        assert call(**kw) == 0, kw

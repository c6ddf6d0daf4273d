"""Host-side checks of the routing entry points: bad arguments are refused
before any launch (fake device addresses, never dereferenced)."""
import pytest

from mxfp8_quantization_moe_amd import _capi, build

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return _capi.load()


def test_capacity(lib):
    cap = lib.mxq_moe_row_capacity
    assert cap(0, 2, 8, 16) == 0
    assert cap(1, 2, 8, 16) == 2 + 2 * 15      # at most two experts have a slot
    assert cap(100, 2, 8, 16) == 200 + 8 * 15
    assert cap(100, 2, 8, 1) == 200
    for bad in ((-1, 2, 8, 1), (1, 0, 8, 1), (1, 9, 8, 1), (1, 33, 64, 1), (1, 2, 4097, 1), (1, 2, 8, 0), (1, 2, 8, 4097),
                (1 << 31, 1, 8, 1), (1 << 30, 2, 8, 1), ((1 << 31) - 1, 1, 8, 16)):
        assert cap(*bad) == -1, bad


def test_route_workspace(lib):
    fn = lib.mxq_moe_route_workspace_bytes
    assert fn(0, 8, 2) == 0 and fn(64, 8, 2) == 0   # one run of tokens
    assert fn(65, 8, 2) > 0
    assert fn(10 ** 7, 8, 2) <= 8 * 8 + 256 * 18 * 4   # never more than 256 runs
    assert fn(64, 8, 9) == -1 and fn(-1, 8, 2) == -1


def test_route_refuses(lib):
    ok = dict(l=A, dt=0, T=100, E=8, sl=8, se=1, mask=0, k=2, renorm=1, align=16, ids=A, w=A, rows=A, lse=A, counts=A,
              offs=A, mean=A, losses=A, live=A, ws=A, bytes=1 << 20)

    def call(**kw):
        return lib.mxq_moe_route(*dict(ok, **kw).values(), None)

    for name in ("l", "ids", "w", "rows", "lse", "counts", "offs", "mean", "losses", "live"):
        assert call(**{name: 0}) == 1, name
    for kw in (dict(dt=2), dict(T=-1), dict(E=0), dict(E=4097), dict(k=0), dict(k=9), dict(renorm=2), dict(align=0),
               dict(sl=-8), dict(l=A + 1), dict(dt=1, l=A + 2), dict(ws=A + 4)):
        assert call(**kw) == 1, kw
    assert call(se=2) == 2
    assert call(bytes=4) == 4 and call(ws=0) == 4


def test_route_backward_refuses(lib):
    ok = dict(l=A, dt=1, T=10, E=8, sl=8, se=1, k=2, renorm=1, ids=A, w=A, lse=A, counts=A, live=A, gw=A, gl=A, dl=A,
              sg=8, sge=1)

    def call(**kw):
        return lib.mxq_moe_route_backward(*dict(ok, **kw).values(), None)

    for name in ("l", "ids", "w", "lse", "counts", "live", "dl"):
        assert call(**{name: 0}) == 1, name
    for kw in (dict(dt=-1), dict(sg=7), dict(dl=A + 2), dict(k=9), dict(sl=-1)):
        assert call(**kw) == 1, kw
    assert call(se=2) == 2 and call(sge=3) == 2
    assert call(T=0) == 0


def test_rows_refuse(lib):
    d = dict(x=A, dt=0, T=10, W=64, sx=64, sxc=1, rows=A, k=2, counts=A, offs=A, E=8, xg=A, cap=20, sg=64, sgc=1)

    def dispatch(**kw):
        return lib.mxq_moe_dispatch(*dict(d, **kw).values(), None)

    for name in ("x", "rows", "counts", "offs", "xg"):
        assert dispatch(**{name: 0}) == 1, name
    for kw in (dict(dt=3), dict(W=-1), dict(cap=-1), dict(cap=1 << 31), dict(sg=63), dict(x=A + 1), dict(k=33), dict(sx=-1)):
        assert dispatch(**kw) == 1, kw
    assert dispatch(sxc=2) == 2 and dispatch(sgc=2) == 2
    assert dispatch(W=0) == 0 and dispatch(cap=0) == 0

    c = dict(yg=A, dt=0, cap=20, W=64, sg=64, sgc=1, rows=A, w=A, k=2, res=A, sr=64, src=1, y=A, sy=64, syc=1, T=10)

    def combine(**kw):
        return lib.mxq_moe_combine(*dict(c, **kw).values(), None)

    for name in ("yg", "rows", "y"):
        assert combine(**{name: 0}) == 1, name
    assert combine(sy=63) == 1 and combine(res=A + 1) == 1 and combine(dt=7) == 1
    assert combine(sgc=2) == 2 and combine(src=2) == 2 and combine(syc=2) == 2
    assert combine(T=0) == 0 and combine(W=0) == 0

    b = dict(dy=A, dt=0, T=10, W=64, sy=64, syc=1, yg=A, sg=64, sgc=1, rows=A, w=A, k=2, counts=A, offs=A, E=8, cap=20,
             dyg=A, sd=64, sdc=1, dw=A)

    def backward(**kw):
        return lib.mxq_moe_combine_backward(*dict(b, **kw).values(), None)

    for name in ("dy", "yg", "rows", "w", "counts", "offs", "dyg", "dw"):
        assert backward(**{name: 0}) == 1, name
    assert backward(sd=63) == 1 and backward(E=0) == 1
    assert backward(syc=2) == 2 and backward(sgc=2) == 2 and backward(sdc=2) == 2
    assert backward(T=0, cap=0) == 0


def test_rows_refuse_widths_past_32_bits(lib):
    for W in ((1 << 30) + 1, (1 << 31) - 1, 1 << 31):
        assert lib.mxq_moe_dispatch(A, 0, 10, W, 0, 1, A, 2, A, A, 8, A, 20, W, 1, None) == 1
        assert lib.mxq_moe_combine(A, 0, 20, W, W, 1, A, A, 2, 0, 0, 1, A, W, 1, 10, None) == 1
        assert lib.mxq_moe_combine_backward(A, 0, 10, W, 0, 1, A, W, 1, A, A, 2, A, A, 8, 20, A, W, 1, A, None) == 1

"""Argument checks of the experts' products' C entry points; no GPU is touched."""
import pytest

from mxfp8_quantization_moe_amd import _capi, build

A = 1 << 20  # a plausible, aligned address; every call here returns before a launch
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return _capi.load()


FORWARD = dict(x=A, rows=100, width=64, sxr=64, sxc=1, w=A, E=3, wide=96, swe=64 * 96, swn=64, swk=1, offs=A, bias=0,
               bdt=1, sbe=96, act=1, gated=0, res=0, srr=96, src=1, y=A, syr=96, syc=1, pre=0, spr=96, spc=1, ws=A, bytes=BIG)
MX = dict(x=A, rows=100, width=64, sxr=64, sxc=1, xs=A, xsr=2, xsb=1, w=A, E=3, wide=96, swe=64 * 96, swn=64, swk=1, wsc=A,
          wse=192, wsn=2, wsb=1, offs=A, bias=0, bdt=1, sbe=96, act=1, gated=0, res=0, srr=96, src=1, y=A, syr=96, syc=1,
          pre=0, spr=96, spc=1, ws=A, bytes=BIG)
BACKWARD = dict(g=A, sgr=96, sgc=1, x=A, rows=100, width=64, sxr=64, sxc=1, w=A, E=3, wide=96, swe=64 * 96, swn=64, swk=1,
                offs=A, pre=A, spr=96, spc=1, act=1, gated=0, dx=A, dxr=64, dxc=1, dw=A, dwe=64 * 96, dwn=64, dwk=1, db=A,
                ws=A, bytes=BIG)


def caller(fn, defaults):
    def call(**kw):
        assert set(kw) <= set(defaults)
        return fn(*dict(defaults, **kw).values(), None)

    return call


COMMON_BAD = (dict(rows=-1), dict(rows=2 ** 31), dict(width=-1), dict(width=65537), dict(wide=-1), dict(wide=65537), dict(E=0),
              dict(E=4097), dict(act=-1), dict(act=4), dict(gated=2), dict(gated=1, wide=95), dict(offs=0), dict(x=0),
              dict(w=0), dict(ws=A + 8))


@pytest.mark.parametrize("name", ["mxq_moe_linear", "mxq_moe_linear_mx", "mxq_moe_linear_backward"])
def test_what_all_refuse(lib, name):
    call = caller(getattr(lib, name), {"mxq_moe_linear": FORWARD, "mxq_moe_linear_mx": MX, "mxq_moe_linear_backward": BACKWARD}[name])
    for kw in COMMON_BAD:
        assert call(**kw) == 1, kw
    for kw in (dict(sxc=2), dict(swk=2)):
        assert call(**kw) == 2, kw


@pytest.mark.parametrize("name,defaults", [("mxq_moe_linear", FORWARD), ("mxq_moe_linear_mx", MX)])
def test_epilogue_refusals(lib, name, defaults):
    call = caller(getattr(lib, name), defaults)
    for kw in (dict(y=0), dict(y=A + 1), dict(syr=95), dict(syr=-1), dict(res=A + 1), dict(res=A, srr=-1), dict(pre=A + 1),
               dict(pre=A, spr=95), dict(bias=A, bdt=2), dict(bias=A + 2), dict(bias=A + 1, bdt=0), dict(bias=A, sbe=-1)):
        assert call(**kw) == 1, kw
    for kw in (dict(syc=2, syr=192), dict(res=A, src=2), dict(pre=A, spc=2)):
        assert call(**kw) == 2, kw
    assert call(rows=0, x=0, y=0) == 0 and call(wide=0, w=0, y=0) == 0


def test_forward_refusals(lib):
    call = caller(lib.mxq_moe_linear, FORWARD)
    for kw in (dict(x=A + 1), dict(w=A + 1), dict(sxr=-1), dict(swn=-1), dict(swe=-1)):
        assert call(**kw) == 1, kw
    # operands that have to be copied first
    need = lib.mxq_moe_linear_workspace_bytes(100, 64, 3, 96, 0)
    assert need >= 2 * 64 * (100 + 3 * 96)
    for kw in (dict(x=A + 2), dict(sxr=65), dict(swn=65, swe=65 * 96), dict(width=63), dict(sxr=0), dict(w=A + 2)):
        for room in (dict(bytes=0), dict(ws=0)):
            assert call(**kw, **room) == 4, kw
    assert call(x=A + 2, w=A + 2, bytes=need - 1) == 4
    # a gated expert's weights of 2 GiB and more
    assert call(gated=1, wide=65536, width=32768, sxr=32768, swn=32768, swe=2 ** 31, E=1, sbe=65536, syr=65536) == 2


def test_mx_refusals(lib):
    call = caller(lib.mxq_moe_linear_mx, MX)
    for kw in (dict(width=48), dict(x=A + 8), dict(w=A + 8), dict(sxr=72), dict(swn=72), dict(swe=8), dict(xs=0), dict(wsc=0),
               dict(xsr=-1), dict(xsb=-1), dict(wse=-1), dict(wsn=-1), dict(wsb=-1), dict(sxr=-16), dict(sxr=1 << 22)):
        assert call(**kw) == 1, kw
    need = lib.mxq_moe_linear_mx_workspace_bytes(4096, 64, 3, 4096, 1)  # rows of two scales: no whole words
    assert need >= 4 * (4096 + 3 * 4096)
    large = dict(rows=4096, wide=4096, syr=4096)
    for kw in (dict(bytes=need - 1), dict(bytes=0), dict(ws=0)):
        assert call(**large, **kw) == 4, kw


def test_backward_refusals(lib):
    call = caller(lib.mxq_moe_linear_backward, BACKWARD)
    for kw in (dict(g=0), dict(g=A + 1), dict(sgr=-1), dict(pre=0), dict(pre=A + 1), dict(spr=-1), dict(dxr=63), dict(dwn=63),
               dict(dwe=64 * 95), dict(dx=A + 1), dict(dw=A + 1), dict(db=A + 2)):
        assert call(**kw) == 1, kw
    for kw in (dict(sgc=2), dict(spc=2), dict(dxc=2, dxr=128), dict(dwk=2, dwn=128, dwe=128 * 96)):
        assert call(**kw) == 2, kw
    need = lib.mxq_moe_linear_backward_workspace_bytes
    assert need(100, 64, 3, 96, 0, 0, 0, 1) == 0
    assert need(100, 64, 3, 96, 1, 0, 0, 1) >= 100 * 96 * 2
    assert need(100, 64, 3, 96, 0, 0, 1, 1) >= 2 * 96 * 4
    assert need(100, 64, 3, 96, 0, 0, 0, 0) >= 2 * (100 * 96 + 100 * 64 + 3 * 96 * 64)
    short = need(100, 64, 3, 96, 1, 0, 1, 1) - 1
    for kw in (dict(bytes=short), dict(bytes=0), dict(ws=0)):
        assert call(**kw) == 4, kw


def test_workspace_queries(lib):
    lin, mx, back = (lib.mxq_moe_linear_workspace_bytes, lib.mxq_moe_linear_mx_workspace_bytes,
                     lib.mxq_moe_linear_backward_workspace_bytes)
    for bad in ((-1, 4, 1, 4), (1, -1, 1, 4), (1, 4, 0, 4), (1, 4, 4097, 4), (1, 4, 1, -1), (1, 65537, 1, 4), (1, 4, 1, 65537)):
        assert lin(*bad, 1) == -1 and mx(*bad, 1) == -1 and back(*bad, 0, 0, 0, 1) == -1, bad
    assert lin(1000, 64, 4, 33, 1) == 0 and lin(1000, 64, 4, 33, 0) > 0 and lin(1000, 63, 4, 33, 1) > 0
    assert mx(1000, 48, 4, 33, 1) == -1 and mx(4096, 128, 4, 4096, 1) == 0 and mx(4096, 128, 4, 4096, 0) > 0
    assert mx(1000, 128, 4, 33, 0) == 0  # small tiles read the scales from where they are
    assert back(10, 8, 2, 7, 0, 1, 0, 1) == -1 and back(10, 8, 2, 8, 4, 0, 0, 1) == -1


def test_few_rows_over_more_columns_than_one_grid_takes(lib):
    """Such a call goes to the tiles, which copy operands of any alignment."""
    assert lib.mxq_moe_linear_workspace_bytes(16, 64, 4096, 2048, 0) == 0
    assert lib.mxq_moe_linear_workspace_bytes(16, 64, 4096, 65536, 0) >= 4096 * 65536 * 64 * 2

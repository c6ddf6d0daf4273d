"""Argument checks of the few-token layer's C entry points; no GPU is touched."""
import pytest

from mxfp8_quantization_moe_amd import _capi, build

A = 1 << 20  # a plausible, aligned address; every call here returns before a launch

ARGS = dict(x=A, T=4, D=64, sxt=64, sxc=1, logits=A, ldt=1, E=8, slt=8, sle=1, mask=0, k=2, renorm=1, H=32, fmt=0, up=A, us=0,
            sue=64 * 64, sur=64, suc=1, suse=128, susr=2, susb=1, bu=0, down=A, ds=0, sde=64 * 32, sdr=32, sdc=1, sdse=64,
            sdsr=1, sdsb=1, bd=0, bdt=1, sbu=64, sbd=64, act=3, gated=1, res=0, srt=64, src=1, y=A, syt=64, syc=1, ws=A,
            bytes=1 << 40)


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return _capi.load()


def test_refusals(lib):
    def call(**kw):
        assert set(kw) <= set(ARGS)
        return lib.mxq_moe_layer(*dict(ARGS, **kw).values(), None)

    for kw in (dict(T=-1), dict(T=65), dict(D=-1), dict(D=65537), dict(H=-1), dict(H=65537), dict(E=0), dict(E=1025), dict(k=0),
               dict(k=9), dict(E=64, k=33), dict(ldt=2), dict(renorm=2), dict(fmt=2), dict(fmt=-1), dict(act=-1), dict(act=4),
               dict(gated=2), dict(ws=A + 8), dict(x=0), dict(x=A + 1), dict(logits=0), dict(logits=A + 2), dict(y=0),
               dict(y=A + 1), dict(syt=63), dict(sxt=-1), dict(slt=-1), dict(res=A + 1), dict(res=A, srt=-1), dict(up=0),
               dict(down=0), dict(up=A + 1), dict(down=A + 1), dict(sue=-1), dict(sdr=-1), dict(bu=A, bdt=2), dict(bd=A + 2),
               dict(bu=A, sbu=-1), dict(bd=A, sbd=-1), dict(H=0, bd=A, sbd=-1)):
        assert call(**kw) == 1, kw
    for kw in (dict(sxc=2), dict(syc=2, syt=128), dict(sle=2), dict(res=A, src=2), dict(suc=2), dict(sdc=2)):
        assert call(**kw) == 2, kw
    mx = dict(fmt=1, us=A, ds=A)
    for kw in (dict(us=0), dict(ds=0), dict(D=48), dict(H=48), dict(up=A + 8), dict(down=A + 8), dict(sur=72), dict(sde=8),
               dict(susr=-1), dict(sdse=-1)):
        assert call(**dict(mx, **kw)) == 1, kw
    assert call(**mx, susb=2) == 2
    need = lib.mxq_moe_layer_workspace_bytes(4, 64, 32, 8, 2)
    for kw in (dict(bytes=need - 1), dict(ws=0)):
        assert call(**kw) == 4, kw
    assert call(T=0) == 0 and call(D=0) == 0


def test_workspace_bytes(lib):
    need = lib.mxq_moe_layer_workspace_bytes
    for bad in ((-1, 4, 4, 4, 1), (65, 4, 4, 4, 1), (1, -1, 4, 4, 1), (1, 4, 65537, 4, 1), (1, 4, 4, 0, 1), (1, 4, 4, 1025, 1),
                (1, 4, 4, 4, 5), (1, 4, 4, 64, 33)):
        assert need(*bad) == -1, bad
    # ids, weights and h in two parts for every slot
    assert need(8, 256, 128, 64, 8) >= 64 * (8 + 2 * 2 * 128)

"""The router against a plain 64-bit form: selection, counts, groups and rows
exactly; weights, losses and gradients within bounds derived from fp32
arithmetic (below), at sizes around the kernels' tiles, with ties, masked
tokens, unavailable experts and strided logits."""
import numpy as np
import pytest
import torch

import moe_reference as ref
import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# fp32 bounds.  exp(x) for |x| <= X carries a relative error of about
# (1 + 1.5 X) 2^-24 (the product x * log2 e is rounded), X <= 24 in these
# inputs: 37 * 2^-24 = 2.2e-6; a sum of E <= 4096 terms in a tree adds
# log2(E) * 2^-24 < 1e-6; a quotient doubles both.  RTOL covers them.
RTOL = 1e-5


def make(T, E, dtype, seed, ties=False, limited=False, masked=False, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    l = 1.5 * torch.randn(T, E, generator=g)
    if ties:  # few distinct values: most rows have equal logits
        l = (l * 2).round() / 2
    if limited:
        l[torch.rand(T, E, generator=g) < 0.6] = -float("inf")
        if T > 2:
            l[T // 2] = -float("inf")
    l = l.to(dtype)
    mask = (torch.rand(T, generator=g) < 0.7) if masked else None
    buf = torch.full((T * (E + pad) + shift + 1,), float("nan"), dtype=dtype)
    view = buf[shift:].as_strided((T, E), (E + pad, 1))
    view.copy_(l)
    dev = buf.to(DEV)[shift:].as_strided((T, E), (E + pad, 1))
    return l.double().numpy(), dev, mask


def check(T, E, k, dtype=torch.float32, renorm=True, align=1, **kw):
    l, dev, mask = make(T, E, dtype, T * 1000 + E, **kw)
    m = None if mask is None else mask.numpy()
    want = ref.route(l, k, m, renorm, align)
    r = mxq.moe_route(dev, k, token_mask=None if mask is None else mask.to(DEV), renormalize=renorm, align=align)
    for name in ("ids", "counts", "offs", "rows"):
        bad = np.argwhere(getattr(r, name).cpu().numpy() != want[name])
        assert not bad.size, (name, len(bad), bad[:5].tolist())
    assert int(r.live) == want["live"]
    assert r.offs.dtype == torch.int32
    for name in ("weights", "mean_prob", "losses"):
        np.testing.assert_allclose(getattr(r, name).double().cpu().numpy(), want[name], rtol=RTOL, atol=1e-30, err_msg=name)
    # lse = log(sum) + max: absolute rounding of the sum and of the result
    np.testing.assert_allclose(r.lse.double().cpu().numpy(), want["lse"], rtol=RTOL, atol=4e-6)

    g = np.random.default_rng(7)
    gw = g.normal(size=(T, k)).astype(np.float32)
    gl = np.array([0.5, 0.25], np.float32)
    for use_w, use_l in ((True, True), (False, True), (True, False)):
        d = mxq.moe_route_backward(dev, r, torch.from_numpy(gw).to(DEV) if use_w else None,
                                   torch.from_numpy(gl).to(DEV) if use_l else None).double().cpu().numpy()
        w = ref.route_backward(want, k, renorm, gw.astype(np.float64) if use_w else None,
                               gl.astype(np.float64) if use_l else np.zeros(2))
        # every term is p times a number below size, each with RTOL
        n = max(want["live"], 1)
        size = np.zeros((T, 1))
        if use_w:
            sel = np.where(want["ids"] >= 0, np.take_along_axis(want["p"], np.maximum(want["ids"], 0), 1), 0).sum(1)
            size += (np.abs(gw).max(1) / np.where(renorm & (sel > 0), sel, 1.0))[:, None] * 4
        if use_l:
            size += gl[0] * E * want["counts"].max() / (n * n * k) * 2
            size += (gl[1] * 2 / n * np.abs(np.where(np.isfinite(want["lse"]), want["lse"], 0)))[:, None]
        tol = RTOL * want["p"] * size + 1e-30
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(w)  # rounded to 8 significant bits
        assert (np.abs(d - w) <= tol).all(), (use_w, use_l, np.abs(d - w).max())


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 129, 1000])
@pytest.mark.parametrize("E,k", [(8, 2), (61, 6)])
def test_token_counts(T, E, k):
    check(T, E, k, masked=T > 64, align=16)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (3, 2), (7, 7), (9, 3), (13, 13), (32, 32), (33, 8), (64, 6), (40, 20), (64, 32), (100, 17), (128, 32), (500, 32), (128, 8),
                                 (129, 32), (200, 5), (256, 8), (257, 1), (384, 6), (512, 10), (700, 4), (1024, 8),
                                 (1500, 3), (4096, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_expert_counts(E, k, dtype):
    check(150, E, k, dtype=dtype, renorm=E % 2 == 0, align=1 + E % 3)


@pytest.mark.parametrize("E,k", [(8, 3), (64, 8), (256, 8), (300, 4)])
def test_ties_go_to_the_lower_expert(E, k):
    check(200, E, k, dtype=torch.bfloat16, ties=True)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(4, 4), (61, 8), (256, 32)])
def test_unavailable_experts_and_masked_tokens(E, k, renorm):
    check(333, E, k, renorm=renorm, limited=True, masked=True, align=32)


@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (5, 3), (8, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_logits(pad, shift, dtype):
    check(100, 64, 4, dtype=dtype, pad=pad, shift=shift)
    check(100, 30, 4, dtype=dtype, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_extreme_logits(dtype):
    """The largest and smallest finite logits, infinitesimal ones and signed
    zeros are ordered and taken like any others."""
    top = torch.finfo(dtype).max
    vals = [top, -top, 0.0, -0.0, 1e-40, -1e-40, 3.0, -float("inf"), -top, 88.0, -88.0, 3.0]
    l = torch.tensor([vals, vals[::-1], [-top] * 12, [-float("inf")] * 11 + [-top]], dtype=dtype)
    want = ref.route(l.double().numpy(), 12)
    for k in (3, 12):
        r = mxq.moe_route(l.to(DEV), k)
        assert np.array_equal(r.ids.cpu().numpy(), want["ids"][:, :k])


def test_many_tokens_take_longer_runs():
    check(16384 + 70, 8, 2, masked=True)      # two rounds per run, a short last run
    check(40000, 4, 1, dtype=torch.bfloat16)


def test_no_tokens_and_no_live_tokens():
    r = mxq.moe_route(torch.empty((0, 5), device=DEV), 2)
    assert r.ids.shape == (0, 2) and int(r.counts.abs().sum()) == 0 and int(r.live) == 0
    assert r.losses.tolist() == [0.0, 0.0] and r.offs.tolist() == [0] * 5
    assert mxq.moe_route_backward(torch.empty((0, 5), device=DEV), r).shape == (0, 5)
    l = torch.full((70, 5), -float("inf"), device=DEV)
    l[3] = float("nan")
    for mask in (None, torch.zeros(70, dtype=torch.bool, device=DEV)):
        x = l if mask is None else torch.randn(70, 5, device=DEV)
        r = mxq.moe_route(x, 2, token_mask=mask, align=16)
        assert (r.ids == -1).all() and (r.rows == -1).all() and (r.weights == 0).all()
        assert r.losses.tolist() == [0.0, 0.0] and r.mean_prob.tolist() == [0.0] * 5
        d = mxq.moe_route_backward(x, r, torch.ones(70, 2, device=DEV), torch.ones(2, device=DEV))
        assert (d == 0).all()


def test_nan_in_a_masked_token_reaches_nothing_and_in_a_live_one_is_not_taken():
    x = torch.randn(40, 16, device=DEV)
    x[5] = float("nan")
    mask = torch.ones(40, dtype=torch.bool, device=DEV)
    mask[5] = False
    r = mxq.moe_route(x, 4, token_mask=mask)
    assert torch.isfinite(r.losses).all() and torch.isfinite(r.weights).all()
    d = mxq.moe_route_backward(x, r, torch.ones(40, 4, device=DEV), torch.ones(2, device=DEV))
    assert torch.isfinite(d).all() and (d[5] == 0).all()
    y = torch.randn(40, 16, device=DEV)
    y[7, 3] = float("nan")
    r = mxq.moe_route(y, 4)
    assert 3 not in r.ids[7].tolist() and (r.ids[7] >= 0).all()
    assert torch.isnan(r.losses).all() and torch.isnan(r.lse[7])


def test_repeated_calls_are_the_same_bits_on_any_stream():
    l, dev, _ = make(5000, 60, torch.bfloat16, 3)
    gw, gl = torch.randn(5000, 6, device=DEV), torch.ones(2, device=DEV)
    first = None
    side = torch.cuda.Stream()
    for stream in (None, None, side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        r = mxq.moe_route(dev, 6, stream=stream)
        d = mxq.moe_route_backward(dev, r, gw, gl, stream=stream)
        torch.cuda.synchronize()
        got = [t.clone() for t in r if torch.is_tensor(t)] + [d]
        if first is not None:
            for a, b in zip(first, got):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        first = first or got


def test_expanded_gradients():
    l, dev, _ = make(50, 12, torch.float32, 4)
    r = mxq.moe_route(dev, 3)
    one = torch.full((1, 1), 0.5, device=DEV)
    a = mxq.moe_route_backward(dev, r, one.expand(50, 3), one.reshape(1).expand(2))
    b = mxq.moe_route_backward(dev, r, one.expand(50, 3).contiguous(), torch.full((2,), 0.5, device=DEV))
    assert torch.equal(a, b)


def test_refusals():
    x = torch.randn(10, 8, device=DEV)
    with pytest.raises(TypeError):
        mxq.moe_route(x.double(), 2)
    with pytest.raises(TypeError):
        mxq.moe_route(x, 2, token_mask=torch.ones(9, dtype=torch.bool, device=DEV))
    with pytest.raises(TypeError):
        mxq.moe_route(x, 2, token_mask=torch.ones(10, device=DEV))
    for k, align in ((0, 1), (9, 1), (2, 0), (2, 1 << 20)):
        with pytest.raises(mxq.MXQError):
            mxq.moe_route(x, k, align=align)
    with pytest.raises(mxq.MXQError):
        mxq.moe_route(torch.randn(8, 10, device=DEV).t(), 2)
    r = mxq.moe_route(x, 2)
    with pytest.raises(TypeError):
        mxq.moe_route_backward(x, r, torch.ones(10, 3, device=DEV))
    with pytest.raises(TypeError):
        mxq.moe_route_backward(x, r, torch.ones(10, 2, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        mxq.moe_route_backward(x[:5], r)

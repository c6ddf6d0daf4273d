"""The mixture-of-experts layer for a few tokens against a plain 64-bit form,
over token counts, experts, odd sizes, formats, masks and strides."""
import math

import pytest
import torch

import linear_reference as ref
import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = 2.0 ** -8
SUM = 2.0 ** -23


def normal(*shape, seed=0, scale=1.0, dtype=torch.bfloat16, pad=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    x = (scale * torch.randn(*shape, generator=g)).to(dtype)
    if not pad and not shift:
        return x.to(DEV)
    ld, n = shape[-1] + pad, math.prod(shape[:-1])
    buf = torch.full((n * ld + shift + 8,), float("nan"), dtype=dtype, device=DEV)
    strides = ((shape[1] * ld,) if len(shape) == 3 else ()) + (ld, 1)
    v = buf[shift:].as_strided(shape, strides)
    v.copy_(x)
    return v


def mx(w):
    q, s = mxq.quantize_mx_rowwise(w.reshape(-1, w.shape[-1]))
    return q.view(torch.uint8).reshape(w.shape).view(torch.float8_e4m3fn), s.reshape(*w.shape[:-1], -1)


def choose(logits, k, mask, renorm):
    """(token, expert, weight) by the definition, ties to the lower expert."""
    out = []
    for t, row in enumerate(logits.double().cpu().tolist()):
        if mask is not None and not mask[t]:
            continue
        order = sorted((e for e in range(len(row)) if row[e] > -math.inf), key=lambda e: (-row[e], e))[:k]
        if not order:
            continue
        top = row[order[0]]
        ex = {e: math.exp(row[e] - top) for e in range(len(row)) if row[e] > -math.inf}
        total = sum(ex[e] for e in order) if renorm else sum(ex.values())
        out += [(t, e, ex[e] / total) for e in order]
    return out


def reference(x, slots, up, down, act, gated, bu, bd, resid):
    """(y, bound) without the rounding of y."""
    T, D = x.shape
    y = torch.zeros(T, D, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(y)
    H = down.shape[2]
    for t, e, s in slots:
        xt = x[t:t + 1]
        h, _, size = ref.forward(xt, up[e:e + 1], None, None if bu is None else bu[e:e + 1], act, gated)
        # sums of x, GELU's cdf, weights from exponentials of fp32 differences,
        # h in two bf16 parts
        dh = (D + 8) * SUM * size + 4e-7 * size + (2.0 ** -16 + 2e-6) * h.abs()
        y[t] += s * (down[e] @ h[0])
        bound[t] += s * (down[e].abs() @ (dh[0] + (H + 40) * SUM * h[0].abs()))
        if bd is not None:
            y[t] += s * bd[e].double()
            bound[t] += 3e-6 * s * bd[e].double().abs()
    # the experts' sums join in up to 64 steps
    bound += 72 * SUM * y.abs()
    if resid is not None:
        y += resid.double()
    return y, bound


def check(T, E, k, D, H, fmt="bf16", act="silu", gated=True, bias=None, resid=True, renorm=True, logits=None, mask=None,
          pad=0, shift=0, seed=0, ldtype=torch.float32):
    x = normal(T, D, seed=seed, pad=pad, shift=shift)
    up = normal(E, 2 * H if gated else H, D, seed=seed + 1, scale=D ** -0.5, pad=pad, shift=shift)
    down = normal(E, D, H, seed=seed + 2, scale=H ** -0.5, pad=pad, shift=shift)
    if logits is None:
        logits = normal(T, E, seed=seed + 3, scale=1.5, dtype=ldtype, pad=pad)
    bu = normal(*up.shape[:2], seed=seed + 4, scale=0.3, dtype=bias) if bias is not None else None
    bd = normal(E, D, seed=seed + 5, scale=0.3, dtype=bias) if bias is not None else None
    r = normal(T, D, seed=seed + 6, pad=pad, shift=shift) if resid else None
    if fmt == "mx":
        u, d = mx(up), mx(down)
        up, down = ref.mx_values(*u), ref.mx_values(*d)
    else:
        u, d = up, down
    y = mxq.moe_layer(x, logits, u, d, k, activation=act, gated=gated, bias_up=bu, bias_down=bd, token_mask=mask,
                      renormalize=renorm, residual=r)
    assert y.shape == x.shape and y.dtype == x.dtype
    want, bound = reference(x.double(), choose(logits, k, mask, renorm), up.double(), down.double(), act, gated, bu, bd, r)
    bad = ~((y.double() - want).abs() <= HALF * want.abs() + 1.01 * bound + 1e-30)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), y[bad][:4].tolist(), want[bad][:4].tolist())
    return y


@pytest.mark.parametrize("fmt", ["bf16", "mx"])
@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 15, 16, 17, 31, 33, 48, 64])
def test_token_counts(T, fmt):
    check(T, 12, 3, 160, 96, fmt)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 1), (64, 8), (65, 4), (256, 8), (257, 6), (1000, 32), (1024, 2)])
def test_experts(E, k):
    for T in (1, 5, 40):
        check(T, E, k, 64, 32)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_epilogues(act, gated):
    check(6, 9, 4, 192, 64, "bf16", act, gated, torch.float32)
    check(20, 9, 4, 192, 64, "mx", act, gated, torch.bfloat16, resid=False, renorm=False)


@pytest.mark.parametrize("D,H", [(1, 1), (7, 5), (16, 33), (31, 257), (33, 8), (130, 300), (1111, 333), (257, 1025)])
@pytest.mark.parametrize("T", [3, 37])
def test_odd_sizes(D, H, T):
    check(T, 7, 2, D, H, bias=torch.float32)
    check(T, 7, 2, D, H, gated=False, act="gelu")


@pytest.mark.parametrize("D,H", [(32, 32), (96, 64), (64, 96), (320, 288), (1056, 544)])
@pytest.mark.parametrize("T", [3, 37])
def test_mx_sizes(D, H, T):
    check(T, 7, 2, D, H, "mx", bias=torch.float32)


def test_every_token_to_the_same_experts():
    logits = torch.zeros(64, 300, device=DEV)
    logits[:, [7, 299, 64]] = torch.tensor([3.0, 2.0, 1.0], device=DEV)
    check(64, 300, 3, 96, 64, logits=logits)
    check(64, 300, 3, 96, 64, "mx", logits=logits)


@pytest.mark.parametrize("fmt", ["bf16", "mx"])
def test_equal_calls_give_equal_bits(fmt):
    """Also of experts with more tokens than one pass of the down product takes."""
    T, E, k, D, H = 64, 6, 4, 2048, 512
    x, logits = normal(T, D), normal(T, E, seed=3, dtype=torch.float32)
    up, down = normal(E, 2 * H, D, seed=1, scale=D ** -0.5), normal(E, D, H, seed=2, scale=H ** -0.5)
    u, d = (mx(up), mx(down)) if fmt == "mx" else (up, down)
    want = mxq.moe_layer(x, logits, u, d, k)
    for _ in range(20):
        assert torch.equal(mxq.moe_layer(x, logits, u, d, k), want)


def test_ties_go_to_the_lower_expert():
    logits = torch.tensor([[0.0, -0.0, 1.0, 1.0, 0.0, -2.0], [5.0] * 6, [-1e30] * 6], device=DEV)
    for k in (1, 3, 4, 6):
        check(3, 6, k, 64, 32, logits=logits)


def test_barred_experts_and_masked_tokens():
    logits = normal(10, 40, seed=9, dtype=torch.float32)
    logits[:, 5:38] = -math.inf
    logits[3] = -math.inf
    logits[4, 1:] = -math.inf
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 0, 1, 1, 0], dtype=torch.bool, device=DEV)
    for fmt in ("bf16", "mx"):
        check(10, 40, 8, 96, 64, fmt, logits=logits, mask=mask, bias=torch.float32)
    y = check(10, 40, 8, 96, 64, logits=logits, mask=torch.zeros_like(mask), resid=False)
    assert not y.any()
    check(10, 40, 8, 96, 64, logits=logits.to(torch.bfloat16), mask=mask.to(torch.uint8), renorm=False)


def test_nan_and_infinite_logits_stay_with_their_token():
    x, up, down = normal(4, 64), normal(8, 64, 64, seed=1), normal(8, 64, 32, seed=2)
    logits = normal(4, 8, seed=3, dtype=torch.float32)
    want = mxq.moe_layer(x, logits, up, down, 2)
    logits[1, 3], logits[2, 0] = float("nan"), float("inf")
    y = mxq.moe_layer(x, logits, up, down, 2)
    assert torch.equal(y[[0, 3]], want[[0, 3]]) and y[1].isnan().all() and y[2].isnan().all()


def test_infinite_weights_stay_infinite():
    """As the sums give it: an expert's infinity reaches its tokens alone, not as NaN."""
    x = torch.ones(3, 64, dtype=torch.bfloat16, device=DEV)
    up, down = torch.ones(2, 32, 64, dtype=torch.bfloat16, device=DEV), torch.ones(2, 64, 32, dtype=torch.bfloat16, device=DEV)
    up[1] = 3e38
    logits = torch.tensor([[1.0, 0.0], [0.0, 1.0], [1.0, 0.0]], device=DEV)
    y = mxq.moe_layer(x, logits, up, down, 1, activation="none", gated=False)
    assert torch.equal(y[0], y[2]) and (y[0] == 2048).all() and (y[1] == math.inf).all()


@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (5, 3), (8, 8)])
def test_strides_and_alignment(pad, shift):
    check(6, 9, 4, 104, 72, pad=pad, shift=shift)
    check(33, 9, 4, 104, 72, pad=pad, shift=shift, ldtype=torch.bfloat16)


def test_repeated_operands():
    """One token for all, one expert's weights for all."""
    x, up, down = normal(1, 64).expand(5, 64), normal(1, 64, 64, seed=1).expand(8, 64, 64), normal(1, 64, 32, seed=2).expand(8, 64, 32)
    logits = normal(5, 8, seed=3, dtype=torch.float32)
    y = mxq.moe_layer(x, logits, up, down, 2)
    assert torch.equal(y, mxq.moe_layer(x.contiguous(), logits, up.contiguous(), down.contiguous(), 2))


def test_no_tokens_no_width_no_hidden():
    new = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    logits = torch.zeros(3, 4, device=DEV)
    assert mxq.moe_layer(new(0, 8), logits[:0], new(4, 8, 8), new(4, 8, 4), 2).shape == (0, 8)
    assert mxq.moe_layer(new(3, 0), logits, new(4, 8, 0), new(4, 0, 4), 2).shape == (3, 0)
    y = mxq.moe_layer(new(3, 8), logits, new(4, 0, 8), new(4, 8, 0), 2, bias_down=new(4, 8), residual=new(3, 8))
    assert (y == 2).all()


def test_refusals():
    new = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    logits = torch.zeros(3, 4, device=DEV)
    ok = dict(x=new(3, 32), logits=logits, up=new(4, 64, 32), down=new(4, 32, 32), top_k=2)
    call = lambda **kw: mxq.moe_layer(**dict(ok, **kw))  # noqa: E731
    call()
    for kw in (dict(x=new(3, 32).float()), dict(x=new(3, 31)), dict(logits=logits[:2]), dict(logits=logits.double()),
               dict(up=new(4, 63, 32)), dict(up=new(3, 64, 32)), dict(down=new(4, 32, 31)), dict(bias_up=new(4, 63)),
               dict(bias_down=new(4, 32), bias_up=new(4, 64).float()), dict(residual=new(3, 31)), dict(up=mx(new(4, 64, 32))),
               dict(token_mask=torch.ones(2, dtype=torch.bool, device=DEV)), dict(token_mask=torch.ones(3, device=DEV))):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(ValueError):
        call(activation="tanh")
    for kw in (dict(top_k=0), dict(top_k=5), dict(x=new(65, 32), logits=torch.zeros(65, 4, device=DEV))):
        with pytest.raises(mxq.MXQError):
            call(**kw)
    with pytest.raises(mxq.MXQError):
        call(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_the_same_as_the_operators_one_by_one():
    """Router, dispatch, the two products and the combine give the same layer."""
    T, E, k, D, H = 40, 16, 4, 256, 128
    x, up, down = normal(T, D), normal(E, 2 * H, D, seed=1, scale=D ** -0.5), normal(E, D, H, seed=2, scale=H ** -0.5)
    logits = normal(T, E, seed=3, dtype=torch.float32)
    y = mxq.moe_layer(x, logits, up, down, k, residual=x)
    r = mxq.moe_route(logits, k, align=16)
    h = mxq.moe_linear(mxq.moe_dispatch(x, r), up, r.offs, activation="silu", gated=True)
    chain = mxq.moe_combine(mxq.moe_linear(h, down, r.offs), r, residual=x)
    # there h and the experts' results are rounded to bf16 too
    assert torch.linalg.vector_norm(y.double() - chain.double()) < 2 * HALF * torch.linalg.vector_norm(chain.double())


@pytest.mark.parametrize("T,fmt", [(1, "bf16"), (8, "mx"), (50, "bf16")])
def test_captured_and_replayed(T, fmt):
    E, k, D, H = 32, 4, 256, 160
    x, logits = normal(T, D), normal(T, E, seed=3, dtype=torch.float32)
    up, down = normal(E, 2 * H, D, seed=1, scale=D ** -0.5), normal(E, D, H, seed=2, scale=H ** -0.5)
    u, d = (mx(up), mx(down)) if fmt == "mx" else (up, down)
    ws = mxq.moe_layer_workspace(T, D, H, E, k)
    call = lambda w=None: mxq.moe_layer(x, logits, u, d, k, residual=x, workspace=w)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call(ws)
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.normal_(generator=g)
        logits.normal_(generator=g)
        want = call().clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    s = torch.cuda.Stream()
    got = mxq.moe_layer(x, logits, u, d, k, residual=x, stream=s)
    s.synchronize()
    assert torch.equal(got, want)

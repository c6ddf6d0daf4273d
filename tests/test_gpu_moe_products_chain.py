"""Router, dispatch, the experts' products, combine and all their gradients run
together: against 64-bit autograd, captured and replayed, and the refusals of
the products' bindings."""
import importlib.util
import os

import pytest
import torch

import linear_reference as ref
import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = 2.0 ** -8  # a rounding to bf16
REST = 2.0 ** -14  # fp32 sums of some hundred terms, exponentials


def normal(*shape, seed=0, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def norm(t):
    return float(torch.linalg.vector_norm(t.detach().double()))


def gain(w):
    """The largest factor by which an expert's product lengthens a row."""
    return max(float(torch.linalg.matrix_norm(m.double(), 2)) for m in w)


def chain(x, logits, up, bias, down, k, c, act="silu"):
    r = mxq.moe_route(logits, k, align=16)
    xg = mxq.moe_dispatch(x, r)
    h, pre = mxq.moe_linear(xg, up, r.offs, bias=bias, activation=act, gated=True, save_pre=True)
    yg = mxq.moe_linear(h, down, r.offs)
    y = mxq.moe_combine(yg, r, residual=x)
    dyg, dw = mxq.moe_combine_backward(c, yg, r)
    dh, ddown, _ = mxq.moe_linear_backward(dyg, h, down, r.offs)
    dxg, dup, dbias = mxq.moe_linear_backward(dh, xg, up, r.offs, pre=pre, activation=act, gated=True, bias=True)
    dx = mxq.moe_dispatch_backward(dxg, r)
    dlogits = mxq.moe_route_backward(logits, r, dw)
    return r, dict(y=y, dx=dx, dup=dup, dbias=dbias, ddown=ddown, dlogits=dlogits)


@pytest.mark.parametrize("T,E,k,D,H", [(1, 3, 1, 64, 32), (70, 5, 2, 48, 40), (300, 16, 4, 256, 128), (41, 8, 3, 77, 51)])
def test_gradients_of_the_chain(T, E, k, D, H):
    """In 2-norms; u = half a step of bf16, |W| the largest singular value.
    Forward: h and its product are rounded, then y.  Backward: dyg, dh, dz, the
    rows' gradients and their sums, and what z's rounding does to the
    derivatives (|act'| <= 1.1, |act''| <= 1/2 with silu)."""
    x, c = normal(T, D), normal(T, D, seed=1)
    logits = normal(T, E, seed=2, dtype=torch.float32)
    up, bias = normal(E, 2 * H, D, seed=3, scale=D ** -0.5), normal(E, 2 * H, seed=4, scale=0.3, dtype=torch.float32)
    down = normal(E, D, H, seed=5, scale=H ** -0.5)
    r, got = chain(x, logits, up, bias, down, k, c)

    leaves = [t.double().requires_grad_() for t in (x, logits, up, bias, down)]
    xr, lr, ur, br, dr = leaves
    w, ids = lr.softmax(1).topk(k, 1)
    assert torch.equal(ids.int(), r.ids)
    w = w / w.sum(1, keepdim=True)
    slots = [(torch.nonzero(ids == e, as_tuple=True)) for e in range(E)]
    parts = {}
    yr = torch.zeros(T, D, dtype=torch.float64, device=DEV)
    for e, (t, j) in enumerate(slots):
        z = xr[t] @ ur[e].t() + br[e]
        h = ref.act(z[:, :H], "silu")[0] * z[:, H:]
        yg = h @ dr[e].t()
        parts[e] = (z, h, yg)
        yr = yr.index_add(0, t, w[t, j][:, None] * yg)
    yr = yr + xr
    (yr * c.double()).sum().backward()

    with torch.no_grad():
        z, h, yg = (torch.cat([parts[e][i] for e in range(E)]) for i in range(3))
        at = [torch.cat(v) for v in zip(*slots)]
        cs = c.double()[at[0]]
        dyg = w[at[0], at[1]][:, None] * cs
        expert = torch.cat([torch.full_like(t, e) for e, (t, _) in enumerate(slots)])
        dh = torch.bmm(dyg[:, None].float(), down.float()[expert].contiguous())[:, 0].double()
        g, v = z[:, :H], z[:, H:]
        y1, slope = ref.act(g, "silu")
        dz = torch.cat([dh * v * slope, dh * y1], 1)
        u = HALF + REST
        e_yg = gain(down) * u * norm(h) + u * norm(yg)
        e_dh = gain(down) * u * norm(dyg) + u * norm(dh)
        most = 1.1 * float(torch.maximum(v.abs(), g.abs()).max())
        e_dz = 1.5 * most * e_dh + 3 * u * norm(torch.cat([dh * v, dh * g], 1)) + u * norm(dz)
        dxg = torch.bmm(dz[:, None].float(), up.float()[expert].contiguous())[:, 0].double()
        e_dxg = gain(up) * e_dz + u * norm(dxg)
        e_dw = float(cs.norm(dim=1).max()) * e_yg + REST * norm(cs) * norm(yg)
        bounds = dict(y=e_yg + u * norm(yr), dx=k ** 0.5 * e_dxg + u * norm(xr.grad - c.double()),
                      ddown=u * (2 * norm(dyg) * norm(h) + norm(dr.grad)), dup=e_dz * norm(x.double()[at[0]]) + u * norm(ur.grad),
                      dbias=len(dz) ** 0.5 * e_dz, dlogits=2 * e_dw)
        wants = dict(y=yr, dx=xr.grad - c.double(), dup=ur.grad, dbias=br.grad, ddown=dr.grad, dlogits=lr.grad)
    for name, want in wants.items():
        off = norm(got[name].double() - want)
        assert off <= 1.05 * bounds[name] + 1e-9, (name, off, bounds[name], norm(want))
        # and far from a gradient that lacks a factor
        if k > 1:
            assert off < 0.1 * norm(want), (name, off, norm(want))


def test_gradients_against_differences():
    """The sum c y along a step of W and of x, both ways from the same bf16 point
    in fp64, is what the kernels' gradients say."""
    rows, D, H, E = 96, 64, 48, 3
    offs = torch.tensor([32, 40, 96], dtype=torch.int32, device=DEV)
    x, w, c = normal(rows, D), normal(E, 2 * H, D, seed=1, scale=D ** -0.5), normal(rows, H, seed=2)
    for name in ("gelu", "silu", "relu"):
        _, pre = mxq.moe_linear(x, w, offs, activation=name, gated=True, save_pre=True)
        dx, dw, _ = mxq.moe_linear_backward(c, x, w, offs, pre=pre, activation=name, gated=True)
        value = lambda a, b: float((ref.forward(a, b, offs.tolist(), None, name, True)[0] * c.double()).sum())  # noqa: E731
        sx, sw = normal(rows, D, seed=3).double(), normal(E, 2 * H, D, seed=4, scale=D ** -0.5).double()
        eps = 1e-5
        for got, base, step, move in ((dx, x, sx, lambda t: value(x.double() + t * sx, w.double())),
                                      (dw, w, sw, lambda t: value(x.double(), w.double() + t * sw))):
            want = (move(eps) - move(-eps)) / (2 * eps)
            have = float((got.double() * step).sum())
            # a few roundings of every product's terms
            size = norm(got) * norm(step)
            assert abs(have - want) <= 4 * HALF * size, (name, have, want, size)


def test_the_chain_captured_and_replayed():
    T, E, k, D, H = 200, 12, 3, 128, 96
    x, c = normal(T, D), normal(T, D, seed=1)
    logits = normal(T, E, seed=2, dtype=torch.float32)
    up, bias = normal(E, 2 * H, D, seed=3, scale=D ** -0.5), normal(E, 2 * H, seed=4, dtype=torch.float32)
    down = normal(E, D, H, seed=5, scale=H ** -0.5)

    def step():
        out = chain(x, logits, up, bias, down, k, c, "gelu")[1]
        few = mxq.moe_layer(x[:20], logits[:20], up, down, k, activation="gelu", bias_up=bias, residual=x[:20])
        xq, xs = mxq.quantize_mx_rowwise(x)
        wq, ws = mxq.quantize_mx_rowwise(up.view(-1, D))
        return list(out.values()) + [few, mxq.moe_linear_mx(xq, xs, wq.view(up.shape)[0], ws.view(E, 2 * H, -1)[0], gated=True)]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, logits, up):
            t.normal_(generator=g)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("width", [1357, 1344])
def test_copies_and_parts_captured_and_replayed(width):
    """Workspaces of the graph's own: odd rows are copied, long sums taken in parts."""
    x, w = normal(92, width), normal(2, 130, width, seed=1, scale=width ** -0.5)
    offs = torch.tensor([40, 90], dtype=torch.int32, device=DEV)

    def step():
        y, pre = mxq.moe_linear(x, w, offs, activation="silu", gated=True, save_pre=True)
        return [y, pre, *mxq.moe_linear_backward(y, x, w, offs, pre=pre, activation="silu", gated=True, bias=True)]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in range(4):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_streams_at_once():
    """Calls that overlap share nothing: each has the bits it has alone."""
    T, E, k, D, H = 64, 6, 3, 512, 256
    x, logits = normal(T, D), normal(T, E, seed=2, dtype=torch.float32)
    up, down = normal(E, 2 * H, D, seed=3, scale=D ** -0.5), normal(E, D, H, seed=5, scale=H ** -0.5)
    offs = torch.tensor([5, 30, 30, 40, 41, 60], dtype=torch.int32, device=DEV)
    square = normal(E, D, D, seed=6, scale=D ** -0.5)
    call = lambda: (mxq.moe_layer(x, logits, up, down, k), mxq.moe_linear(x[:, :511], up[:, :, :511], offs, gated=True),  # noqa: E731
                    mxq.moe_linear_backward(x, x, square, offs, bias=True))
    flat = lambda v: [t for o in v for t in (o if isinstance(o, tuple) else (o,)) if t is not None]  # noqa: E731
    want = flat(call())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(flat(call()))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_refusals():
    new = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    offs = torch.tensor([3, 6], dtype=torch.int32, device=DEV)
    ok = dict(x=new(6, 32), w=new(2, 8, 32), offs=offs)
    call = lambda **kw: mxq.moe_linear(**dict(ok, **kw))  # noqa: E731
    call(bias=new(2, 8), residual=new(6, 8))
    for kw in (dict(x=new(6, 32).float()), dict(x=new(6, 31)), dict(x=new(6)), dict(w=new(2, 8, 32).float()), dict(w=new(32)),
               dict(w=new(2, 8, 32).cpu()), dict(offs=None), dict(offs=offs.long()), dict(offs=offs[:1]), dict(offs=offs.cpu()),
               dict(bias=new(2, 7)), dict(bias=new(2, 8).half()), dict(bias=new(2, 16)[:, ::2]), dict(residual=new(6, 7)),
               dict(residual=new(6, 8).float()), dict(w=new(2, 7, 32), gated=True), dict(residual=new(6, 8), gated=True)):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(ValueError):
        call(activation="swish")
    for kw in (dict(x=new(32, 6).t()), dict(w=new(2, 32, 8).transpose(1, 2)), dict(residual=new(8, 6).t())):
        with pytest.raises(mxq.MXQError):
            call(**kw)
    back = dict(ok, grad_y=new(6, 8))
    call = lambda **kw: mxq.moe_linear_backward(**dict(back, **kw))  # noqa: E731
    call(bias=True)
    for kw in (dict(grad_y=new(6, 7)), dict(grad_y=new(6, 8).float()), dict(activation="gelu"), dict(gated=True, grad_y=new(6, 4)),
               dict(activation="gelu", pre=new(6, 7)), dict(offs=None), dict(w=new(2, 7, 32), gated=True, grad_y=new(6, 3))):
        with pytest.raises(TypeError):
            call(**kw)
    f8 = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn, device=DEV)  # noqa: E731
    u8 = lambda *s: torch.full(s, 127, dtype=torch.uint8, device=DEV)  # noqa: E731
    mx = dict(x=f8(6, 64), x_scales=u8(6, 2), w=f8(2, 8, 64), w_scales=u8(2, 8, 2), offs=offs)
    call = lambda **kw: mxq.moe_linear_mx(**dict(mx, **kw))  # noqa: E731
    assert not call().any()
    for kw in (dict(x=new(6, 64)), dict(x_scales=u8(6, 1)), dict(x_scales=u8(6, 2).int()), dict(w_scales=u8(2, 8, 1)),
               dict(w=f8(2, 8, 32)), dict(x=f8(6, 48), w=f8(2, 8, 48)), dict(offs=offs[:1])):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(mxq.MXQError):
        call(x=f8(6 * 64 + 1)[1:].view(6, 64))


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_train_step.py")
    spec = importlib.util.spec_from_file_location("moe_train_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("activation", ["none", "relu"])
def test_the_examples_products(example, activation):
    """Their values are those of the quantized operands, their gradients the
    formula's at the saved z."""
    offs = torch.tensor([32, 32, 96], dtype=torch.int32, device=DEV)
    x, w, c = normal(128, 64).requires_grad_(), normal(3, 96, 64, seed=1).requires_grad_(), normal(128, 96, seed=2)
    y = example.ExpertProducts.apply(x, w, offs, activation)
    (y * c).sum().backward()
    xv = ref.mx_values(*mxq.quantize_mx_rowwise(x.detach()))
    wq, ws = mxq.quantize_mx_rowwise(w.detach().view(-1, 64))
    want, _, size = ref.forward(xv, ref.mx_values(wq, ws).view(3, 96, 64), offs.tolist(), None, activation)
    assert ((y.double() - want).abs() <= HALF * want.abs() + 2.0 ** -9 * size + 1e-30).all()
    # relu: z, kept in bf16, is positive where y is
    dz = c.double() if activation == "none" else torch.where(y > 0, c, 0.0).double()
    for e, (lo, hi) in enumerate(((0, 32), (32, 32), (32, 96))):
        gx, gw = dz[lo:hi] @ w[e].double(), dz[lo:hi].t() @ x[lo:hi].double()
        assert ((x.grad[lo:hi].double() - gx).abs() <= HALF * gx.abs() + 2.0 ** -14 * (dz[lo:hi].abs() @ w[e].double().abs()) + 1e-30).all()
        assert ((w.grad[e].double() - gw).abs() <= HALF * gw.abs() + 2.0 ** -14 * (dz[lo:hi].abs().t() @ x[lo:hi].double().abs()) + 1e-30).all()
    assert not x.grad[96:].any()


def test_the_example_decodes(example):
    layer = example.MoeLayer(64, 128, 4, 2)
    x = normal(16, 64)
    y = layer.decode(x)
    assert y.shape == x.shape and y.isfinite().all()

"""The operators together: the example's layer learns, and its gradients are
those of the same layer in plain torch."""
import importlib.util
import os

import pytest
import torch

import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_train_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_train_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_layer_learns(example):
    h = example.train(steps=30, tokens=512, width=64, hidden=128, experts=4, verbose=False)
    first, last = h[0], h[-1]
    assert all(map(lambda v: v == v, sum(h, [])))
    assert last[0] < 0.5 * first[0], (first, last)


def test_gradients_of_the_chain(example):
    """Router, dispatch and combine as autograd functions against the same
    computation by indexing, in fp32, one linear expert each."""
    T, W, E, k = 70, 48, 5, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    x0 = torch.randn(T, W, generator=g, device="cuda")
    router0 = torch.randn(E, W, generator=g, device="cuda") * 0.3
    scale0 = torch.randn(E, W, generator=g, device="cuda")
    c = torch.randn(T, W, generator=g, device="cuda")

    def leaves():
        return [t.clone().requires_grad_() for t in (x0, router0, scale0)]

    x, router, scale = leaves()
    box = []
    weights, losses = example.Route.apply(x @ router.t(), k, 8, box)
    route = box[0]
    xg = example.Dispatch.apply(x, route)
    rows = torch.arange(xg.shape[0], device="cuda")
    expert = torch.searchsorted(route.offs, rows, right=True).clamp(max=E - 1)
    y = example.Combine.apply(xg * scale[expert], weights, x, route)
    ((y * c).sum() + 3.0 * losses[0] + 0.5 * losses[1]).backward()

    xr, rr, sr = leaves()
    logits = xr @ rr.t()
    p = logits.softmax(1)
    w, ids = p.topk(k, 1)
    w = w / w.sum(1, keepdim=True)
    yr = xr + (w[:, :, None] * xr[:, None, :] * sr[ids]).sum(1)
    counts = torch.nn.functional.one_hot(ids, E).sum((0, 1))
    bal = E * (counts / (T * k) * p.mean(0)).sum()
    z = logits.logsumexp(1).square().mean()
    ((yr * c).sum() + 3.0 * bal + 0.5 * z).backward()
    assert torch.equal(ids.int(), route.ids)
    torch.testing.assert_close(y, yr, rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(losses, torch.stack([bal, z]), rtol=1e-4, atol=1e-5)
    for got, want in ((x, xr), (router, rr), (scale, sr)):
        torch.testing.assert_close(got.grad, want.grad, rtol=1e-3, atol=1e-3)


def test_the_groups_feed_the_quantizers():
    """dispatch's rows and group ends are what the jagged quantizers take."""
    T, W, E, k = 300, 64, 6, 2
    x = torch.randn(T, W, device="cuda").to(torch.bfloat16)
    r = mxq.moe_route(torch.randn(T, E, device="cuda"), k, align=16)
    xg = mxq.moe_dispatch(x, r)
    q, s = mxq.quantize_jagged_colwise(xg, r.offs)
    ends = [0] + r.offs.tolist()
    for e in range(E):
        part = xg[ends[e]:ends[e + 1]].float()
        if len(part):
            # one IEEE division on the CPU (torch's 448.0 / t multiplies by a reciprocal)
            want = torch.div(torch.tensor(448.0), part.abs().amax(0).clamp(min=1e-12).cpu())
            torch.testing.assert_close(s[e].cpu(), want, rtol=0, atol=0)


def test_a_captured_step_replays():
    """Router, dispatch, combine and their gradients and the Newton-Schulz
    update in one graph: each replay, with eager work and a synchronization in
    between, gives the eager call's bits."""
    T, W, E, k = 600, 96, 24, 4
    x = torch.randn(T, W, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, device="cuda")
    gw, gl = torch.randn(T, k, device="cuda"), torch.ones(2, device="cuda")
    m = torch.randn(2, 200, 130, device="cuda")

    def step():
        r = mxq.moe_route(logits, k, align=16)
        xg = mxq.moe_dispatch(x, r)
        y = mxq.moe_combine(xg, r, residual=x)
        dyg, dw = mxq.moe_combine_backward(y, xg, r)
        return [xg, y, dyg, dw, mxq.moe_dispatch_backward(dyg, r), mxq.moe_route_backward(logits, r, gw, gl),
                mxq.muon_orthogonalize(m)] + [t for t in r if torch.is_tensor(t)]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        logits.normal_(generator=g)
        x.normal_(generator=g)
        m.normal_(generator=g)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)

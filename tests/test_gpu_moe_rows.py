"""Dispatch, combine and their gradients against plain 64-bit forms, over
types, widths off the 16-byte pieces, strides, empty slots, padded groups and
the rows that belong to no group."""
import numpy as np
import pytest
import torch

import moe_reference as ref
import mxfp8_quantization_moe_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# one rounding to the output type after fp32 sums of at most 33 terms: the
# sum's error is below 33 * 2^-24 of the terms' magnitudes
ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}


def plan(T, E, k, align, seed, empty=0.0, dead_experts=()):
    """A route whose slots were drawn at random, in tensors on the device."""
    g = np.random.default_rng(seed)
    open_ = [e for e in range(E) if e not in dead_experts]
    ids = np.stack([g.choice(open_, k, replace=False) for _ in range(T)]) if T else np.zeros((0, k), int)
    ids = np.where(g.random((T, k)) < empty, -1, ids)
    counts = np.array([(ids == e).sum() for e in range(E)])
    ends = np.cumsum((counts + align - 1) // align * align)
    nxt = (ends - (counts + align - 1) // align * align).copy()
    rows = np.full((T, k), -1)
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                rows[t, j] = nxt[ids[t, j]]
                nxt[ids[t, j]] += 1
    w = np.where(ids >= 0, g.random((T, k)), 0).astype(np.float32)
    i32 = lambda a: torch.from_numpy(a.astype(np.int32)).to(DEV)  # noqa: E731
    return rows, w, mxq.MoeRoute(ids=i32(ids), weights=torch.from_numpy(w).to(DEV), rows=i32(rows), counts=i32(counts),
                                 offs=i32(ends), align=align)


def rows_of(n, W, dtype, seed, pad=0, shift=0):
    """(n, W) rows with a row stride of W + pad, `shift` elements off, in a
    buffer of NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, W, generator=g).to(dtype)
    buf = torch.full((n * (W + pad) + shift + 1,), float("nan"), dtype=dtype, device=DEV)
    v = buf[shift:].as_strided((n, W), (W + pad, 1))
    v.copy_(x)
    return x.double().numpy(), v


def near(got, want, size, dtype, what):
    got = got.double().cpu().numpy()
    tol = ULP[dtype] * np.abs(want) + 40 * 2.0 ** -24 * size + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:5].tolist())


def check(T, E, k, W, dtype, align=1, empty=0.0, dead=(), pad=0, shift=0, residual=False):
    rows, w, r = plan(T, E, k, align, T * 31 + W, empty, dead)
    cap = mxq.moe_row_capacity(T, k, E, align)
    x, xd = rows_of(T, W, dtype, 1, pad, shift)
    xg = mxq.moe_dispatch(xd, r)
    assert xg.shape == (cap, W)
    assert np.array_equal(xg.double().cpu().numpy(), ref.dispatch(x, rows, cap)), "dispatch"

    yg, ygd = rows_of(cap, W, dtype, 2, pad, shift)
    if (rows >= 0).sum() < cap:  # what no slot names may hold anything
        unused = np.setdiff1d(np.arange(cap), rows[rows >= 0])
        ygd[torch.from_numpy(unused).to(DEV)] = float("nan")
    size = ref.combine(np.abs(yg), rows, np.abs(w))
    res, resd = rows_of(T, W, dtype, 3, pad, shift) if residual else (None, None)
    near(mxq.moe_combine(ygd, r, residual=resd), ref.combine(yg, rows, w, res),
         size + (0 if res is None else np.abs(res)), dtype, "combine")
    near(mxq.moe_dispatch_backward(ygd, r), ref.combine(yg, rows, None), ref.combine(np.abs(yg), rows, None), dtype,
         "dispatch backward")

    dy, dyd = rows_of(T, W, dtype, 4, pad, shift)
    dyg, dw = mxq.moe_combine_backward(dyd, ygd, r)
    wyg, wdw = ref.combine_backward(dy, yg, rows, w.astype(np.float64))
    near(dyg, wyg, np.abs(wyg), dtype, "grad_yg")
    # a dot product of W terms in a tree of depth log2: the terms' magnitudes
    # times (W / (64 lanes) + 6 + 4) roundings
    sizes = ref.combine_backward(np.abs(dy), np.abs(yg), rows, w.astype(np.float64))[1]
    assert (np.abs(dw.double().cpu().numpy() - wdw) <= (W / 64 + 12) * 2.0 ** -24 * sizes + 1e-30).all(), "grad_weights"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [1, 3, 4, 7, 8, 9, 63, 64, 200, 511, 512, 513, 1024, 1111, 2048, 2056, 4100])
def test_widths(W, dtype):
    check(37, 5, 2, W, dtype, align=16, residual=W % 2 == 1)


@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 8, 9, 17, 32])
@pytest.mark.parametrize("W", [136, 2304])
def test_slots(k, W):
    check(29, 40, k, W, torch.bfloat16, align=3, empty=0.1, residual=True)
    check(29, 40, k, W, torch.float32, align=1, empty=0.1)


@pytest.mark.parametrize("T", [1, 2, 4, 5, 100])
def test_token_counts(T):
    check(T, 16, 4, 768, torch.bfloat16, align=32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (5, 3), (8, 8)])
def test_strides_and_alignment(pad, shift, dtype):
    check(33, 6, 3, 520, dtype, align=4, pad=pad, shift=shift, residual=True)
    check(33, 6, 3, 5, dtype, align=4, pad=pad, shift=shift, residual=True)


def test_empty_slots_and_groups():
    check(50, 8, 2, 300, torch.bfloat16, align=16, empty=0.5, dead=(0, 3, 7))
    check(50, 8, 2, 300, torch.bfloat16, align=16, empty=1.0, residual=True)
    check(50, 8, 2, 300, torch.float32, align=1, empty=1.0)


def test_no_tokens():
    r = mxq.moe_route(torch.empty((0, 4), device=DEV), 2)
    x = torch.empty((0, 64), device=DEV)
    assert mxq.moe_dispatch(x, r).shape == (0, 64)
    yg = torch.empty((0, 64), device=DEV)
    assert mxq.moe_combine(yg, r).shape == (0, 64)
    assert mxq.moe_combine_backward(x, yg, r)[1].shape == (0, 2)


def test_nothing_outside_the_buffer_is_written():
    """The C entry on a buffer inside a larger one: rows before and after it,
    and the gap between its rows, keep their bytes."""
    T, E, k, W, cap, ld = 21, 4, 2, 100, 21 * 2 + 4 * 15, 112
    rows, w, r = plan(T, E, k, 16, 5)
    x, xd = rows_of(T, W, torch.float32, 1)
    buf = torch.full((cap + 2, ld), 77.0, device=DEV)
    code = mxq.mxq_moe_dispatch(xd.data_ptr(), mxq.MXQ_F32, T, W, W, 1, r.rows.data_ptr(), k, r.counts.data_ptr(),
                                r.offs.data_ptr(), E, buf[1].data_ptr(), cap, ld, 1, None)
    assert code == 0
    torch.cuda.synchronize()
    assert np.array_equal(buf[1:-1, :W].double().cpu().numpy(), ref.dispatch(x, rows, cap))
    assert (buf[0] == 77).all() and (buf[-1] == 77).all() and (buf[:, W:] == 77).all()


def test_rows_outside_the_buffer_are_empty_slots():
    T, E, k, W = 16, 4, 2, 64
    rows, w, r = plan(T, E, k, 1, 6)
    bad = r.rows.clone()
    bad[3, 1], bad[5, 0] = 1 << 30, -7
    rows[3, 1] = rows[5, 0] = -1
    yg, ygd = rows_of(T * k, W, torch.float32, 2)
    near(mxq.moe_combine(ygd, r._replace(rows=bad)), ref.combine(yg, rows, w), ref.combine(np.abs(yg), rows, w),
         torch.float32, "combine")
    dw = mxq.moe_combine_backward(ygd[:T], ygd, r._replace(rows=bad))[1]
    assert float(dw[3, 1]) == 0 and float(dw[5, 0]) == 0


def test_expanded_and_transposed_gradients():
    rows, w, r = plan(20, 4, 2, 1, 8)
    yg, ygd = rows_of(40, 96, torch.float32, 2)
    one = torch.ones((), device=DEV)
    flat = torch.randn(96, 20, device=DEV)
    for dy in (one.expand(20, 96), torch.randn(96, device=DEV).expand(20, 96), flat.t()):
        a, aw = mxq.moe_combine_backward(dy, ygd, r)
        b, bw = mxq.moe_combine_backward(dy.contiguous(), ygd, r)
        assert torch.equal(a, b) and torch.equal(aw, bw)
    g = torch.randn(96, 40, device=DEV)
    assert torch.equal(mxq.moe_dispatch_backward(g.t(), r), mxq.moe_dispatch_backward(g.t().contiguous(), r))
    assert torch.equal(mxq.moe_dispatch_backward(one.expand(40, 96), r), torch.full((20, 96), 2.0, device=DEV))


def test_gradients_match_differences():
    """fp32 kernels on values with few bits: every product and sum is exact,
    and so are the difference quotients of a step of one."""
    g = torch.Generator().manual_seed(9)
    T, E, k, W = 12, 5, 2, 40
    rows, w, r = plan(T, E, k, 8, 10)
    cap = mxq.moe_row_capacity(T, k, E, 8)
    w4 = torch.randint(1, 5, (T, k), generator=g).float().to(DEV)
    r = r._replace(weights=w4)
    yg = torch.randint(-4, 5, (cap, W), generator=g).float().to(DEV)
    c = torch.randint(-4, 5, (T, W), generator=g).float().to(DEV)
    f = lambda y_, r_: float((mxq.moe_combine(y_, r_) * c).sum())  # noqa: E731
    dyg, dw = mxq.moe_combine_backward(c, yg, r)
    base = f(yg, r)
    for row, col in ((0, 0), (3, 39), (cap - 1, 7), (9, 20)):
        y2 = yg.clone()
        y2[row, col] += 1
        assert f(y2, r) - base == float(dyg[row, col])
    for t, j in ((0, 0), (5, 1), (11, 0)):
        w2 = w4.clone()
        w2[t, j] += 1
        assert f(yg, r._replace(weights=w2)) - base == float(dw[t, j])
    x = torch.randint(-4, 5, (T, W), generator=g).float().to(DEV)
    h = torch.randint(-4, 5, (cap, W), generator=g).float().to(DEV)
    dx = mxq.moe_dispatch_backward(h, r)
    base = float((mxq.moe_dispatch(x, r) * h).sum())
    for t, col in ((0, 0), (7, 33)):
        x2 = x.clone()
        x2[t, col] += 1
        assert float((mxq.moe_dispatch(x2, r) * h).sum()) - base == float(dx[t, col])


def test_offsets_past_32_bits():
    """A grouped buffer of more than 2^32 bytes and 2^31 elements: rows at
    its end are reached."""
    T, k, W = 300000, 1, 8192
    rows = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV).reshape(T, 1)
    r = mxq.MoeRoute(weights=torch.full((T, 1), 0.5, device=DEV), rows=rows,
                     counts=torch.tensor([T], dtype=torch.int32, device=DEV),
                     offs=torch.tensor([T], dtype=torch.int32, device=DEV), align=1)
    x = torch.randint(-8, 8, (T, 1), device=DEV).to(torch.bfloat16).expand(T, W) + torch.arange(
        W, device=DEV).remainder(4).to(torch.bfloat16)
    assert x.numel() > 2 ** 31
    xg = mxq.moe_dispatch(x, r)
    assert torch.equal(xg, x.flip(0))
    assert torch.equal(mxq.moe_combine(xg, r), x * 0.5)
    dyg, dw = mxq.moe_combine_backward(x, xg, r)
    assert torch.equal(dyg, xg * 0.5)
    assert torch.equal(dw[:, 0], x.float().square_().sum(1))


def test_refusals():
    rows, w, r = plan(10, 4, 2, 1, 11)
    x = torch.randn(10, 16, device=DEV)
    with pytest.raises(TypeError):
        mxq.moe_dispatch(x.half(), r)
    with pytest.raises(TypeError):
        mxq.moe_dispatch(x[:9], r)
    with pytest.raises(TypeError):
        mxq.moe_dispatch(x, r._replace(rows=r.rows.long()))
    with pytest.raises(TypeError):
        mxq.moe_dispatch(x, r._replace(counts=r.counts[:3]))
    with pytest.raises(mxq.MXQError):
        mxq.moe_dispatch(torch.randn(16, 10, device=DEV).t(), r)
    with pytest.raises(mxq.MXQError):
        mxq.moe_dispatch(x, r._replace(align=0))
    yg = torch.randn(20, 16, device=DEV)
    with pytest.raises(TypeError):
        mxq.moe_combine(yg, r, residual=x.bfloat16())
    with pytest.raises(TypeError):
        mxq.moe_combine(yg, r, residual=x[:, :8])
    with pytest.raises(TypeError):
        mxq.moe_combine_backward(x, yg, r._replace(weights=None))
    with pytest.raises(TypeError):
        mxq.moe_combine_backward(x[:, :8], yg, r)


def test_a_gradient_that_is_copied_first_is_copied_on_the_calls_stream():
    # a transposed gradient gets its copy behind its producer, on the stream given
    torch.manual_seed(5)
    r = mxq.moe_route(torch.randn(500, 8, device=DEV), 2)
    src = torch.randn(64, 1000, device=DEV)
    want = mxq.moe_dispatch_backward(src.t().contiguous(), r)
    grad = torch.zeros(64, 1000, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
        grad.copy_(src)
    got = mxq.moe_dispatch_backward(grad.t(), r, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)

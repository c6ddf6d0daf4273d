"""Mixture-of-experts routing around the quantized grouped products: the
router with its losses and gradients, and the dispatch of token rows into the
expert groups that the quantizers read (``offs``) and back.

Tensor-level binding over the C ABI in ``include/mxq.h`` like the rest of the
package: shapes and types are checked, outputs allocated with torch, device
pointers and the HIP stream forwarded.  With a ``stream`` the outputs are
allocated on that stream.
"""
from __future__ import annotations

from typing import Any, NamedTuple

from . import MXQError, _check, _torch
from ._capi import (MXQ_BF16, MXQ_ERR_INVALID_ARG, MXQ_F32, mxq_moe_combine, mxq_moe_combine_backward,
                    mxq_moe_dispatch, mxq_moe_route, mxq_moe_route_backward, mxq_moe_route_workspace_bytes,
                    mxq_moe_row_capacity)


class MoeRoute(NamedTuple):
    """What the router decides, as device tensors (see mxq_moe_route in
    ``include/mxq.h``): ``ids`` and ``weights`` (tokens, top_k), ``rows``
    (tokens, top_k) the row of each slot in the grouped buffer, ``counts`` and
    ``offs`` (num_experts,), ``mean_prob`` (num_experts,), ``losses`` (2,)
    balance and z, ``lse`` (tokens,), ``live`` (1,).  ``align`` and
    ``renormalize`` are the call's arguments.  The dispatch and combine calls
    need ``weights``, ``rows``, ``counts``, ``offs`` and ``align`` alone, so
    another router's results can be wrapped too."""
    ids: Any = None
    weights: Any = None
    rows: Any = None
    counts: Any = None
    offs: Any = None
    mean_prob: Any = None
    losses: Any = None
    lse: Any = None
    live: Any = None
    align: int = 1
    renormalize: bool = True


def _run(t, stream, call):
    """``call(stream handle)`` with t's device current and, given a stream,
    with that stream as torch's current one, so that what the call allocates
    belongs to the stream that uses it."""
    torch = _torch()
    if stream is None:
        index = t.device.index
        if torch.cuda.current_device() == index:
            # the handle without a Stream object around it: 0.2 us against 3
            return call(torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(t.device):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        if not hasattr(stream, "cuda_stream"):
            stream = (torch.cuda.ExternalStream(int(stream), device=t.device) if int(stream)
                      else torch.cuda.default_stream(t.device))
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _dtype(t, ndim: int, name: str) -> int:
    torch = _torch()
    if t.dim() == ndim and t.is_cuda:
        dtype = t.dtype
        if dtype is torch.bfloat16:
            return MXQ_BF16
        if dtype is torch.float32:
            return MXQ_F32
    raise TypeError(f"{name} must be a {ndim}-D bfloat16 or float32 CUDA tensor, got {t.dtype} "
                    f"{tuple(t.shape)} on {t.device}")


def _same(t, like, shape, name: str) -> None:
    if t.dtype is not like.dtype or t.shape != shape or t.device != like.device:
        raise TypeError(f"{name} must be a {like.dtype} tensor of shape {tuple(shape)} on {like.device}, got "
                        f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _plain(t, dtype, shape, device, name: str) -> None:
    if t is not None and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    got = "None" if t is None else f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}"
    raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got {got}")


def _unit(t):
    """A gradient as autograd may hand it over (an expanded scalar, a
    transposed view): copied if its last dim has no unit stride.  To be called
    within _run, so that the copy is made on the call's stream."""
    return t if t.stride(-1) == 1 and min(t.stride()) >= 0 else t.contiguous()


def moe_row_capacity(tokens: int, top_k: int, num_experts: int, align: int = 1) -> int:
    """Rows of a grouped buffer that holds every group whatever the router
    picks: tokens * top_k plus align - 1 for each expert that can have one."""
    n = mxq_moe_row_capacity(tokens, top_k, num_experts, align)
    if n < 0:
        raise MXQError(MXQ_ERR_INVALID_ARG, "mxq_moe_row_capacity")
    return n


def moe_route(logits, top_k: int, *, token_mask=None, renormalize: bool = True, align: int = 1, stream=None):
    """Routes tokens by their ``logits`` (tokens, num_experts), bf16 or fp32:
    softmax, the ``top_k`` largest (ties to the lower expert; -inf is never
    taken), counts, group ends (each group's rows rounded up to a multiple of
    ``align``), the balance and z losses.  ``token_mask``: bool or uint8
    (tokens,), false for tokens that take part in nothing.  Returns a
    ``MoeRoute``; nothing is read back to the host."""
    torch = _torch()
    dt = _dtype(logits, 2, "logits")
    T, E = logits.shape
    dev = logits.device
    mask = 0
    if token_mask is not None:
        if token_mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"token_mask must be a bool or uint8 tensor, got {token_mask.dtype}")
        _plain(token_mask, token_mask.dtype, (T,), dev, "token_mask")
        mask = token_mask.data_ptr()
    k = int(top_k)
    need = mxq_moe_route_workspace_bytes(T, E, k)
    if need < 0:
        raise MXQError(MXQ_ERR_INVALID_ARG, "mxq_moe_route")

    def call(st):
        slots = T * k
        ints = torch.empty(2 * slots + 2 * E + 1, dtype=torch.int32, device=dev)
        floats = torch.empty(slots + T + E + 2, dtype=torch.float32, device=dev)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        ids, rows, counts, offs, live = ints.split((slots, slots, E, E, 1))
        weights, lse, mean_prob, losses = floats.split((slots, T, E, 2))
        p, f = ints.data_ptr(), floats.data_ptr()
        code = mxq_moe_route(
            logits.data_ptr(), dt, T, E, logits.stride(0), logits.stride(1), mask, k, int(bool(renormalize)),
            int(align), p, f, p + 4 * slots, f + 4 * slots, p + 8 * slots, p + 4 * (2 * slots + E),
            f + 4 * (slots + T), f + 4 * (slots + T + E), p + 8 * (slots + E), ws.data_ptr() if need else 0, need, st)
        _check(code, "mxq_moe_route")
        return MoeRoute(ids.view(T, k), weights.view(T, k), rows.view(T, k), counts, offs, mean_prob, losses, lse,
                        live, int(align), bool(renormalize))

    return _run(logits, stream, call)


def moe_route_backward(logits, route: MoeRoute, grad_weights=None, grad_losses=None, *, stream=None):
    """Gradient of ``route.weights`` and ``route.losses`` with respect to the
    ``logits`` given to ``moe_route``, in their type.  ``grad_weights``
    (tokens, top_k) fp32 and ``grad_losses`` (2,) fp32 on the device, each may
    be None."""
    torch = _torch()
    dt = _dtype(logits, 2, "logits")
    T, E = logits.shape
    dev = logits.device
    k = route.ids.shape[-1] if route.ids is not None and route.ids.dim() == 2 else 0
    _plain(route.ids, torch.int32, (T, k), dev, "route.ids")
    _plain(route.weights, torch.float32, (T, k), dev, "route.weights")
    _plain(route.lse, torch.float32, (T,), dev, "route.lse")
    _plain(route.counts, torch.int32, (E,), dev, "route.counts")
    _plain(route.live, torch.int32, (1,), dev, "route.live")

    def call(st):
        gw = gl = None
        if grad_weights is not None:
            gw = grad_weights.contiguous()
            _plain(gw, torch.float32, (T, k), dev, "grad_weights")
        if grad_losses is not None:
            gl = grad_losses.contiguous()
            _plain(gl, torch.float32, (2,), dev, "grad_losses")
        out = torch.empty((T, E), dtype=logits.dtype, device=dev)
        code = mxq_moe_route_backward(
            logits.data_ptr(), dt, T, E, logits.stride(0), logits.stride(1), k, int(route.renormalize),
            route.ids.data_ptr(), route.weights.data_ptr(), route.lse.data_ptr(), route.counts.data_ptr(),
            route.live.data_ptr(), 0 if gw is None else gw.data_ptr(), 0 if gl is None else gl.data_ptr(),
            out.data_ptr(), E, 1, st)
        _check(code, "mxq_moe_route_backward")
        return out

    return _run(logits, stream, call)


def _plan(route, tokens: int, dev):
    i32 = _torch().int32
    rows, offs = route.rows, route.offs
    k = rows.shape[-1] if rows is not None and rows.dim() == 2 else 0
    _plain(rows, i32, (tokens, k), dev, "route.rows")
    E = offs.numel() if offs is not None else 0
    _plain(offs, i32, (E,), dev, "route.offs")
    _plain(route.counts, i32, (E,), dev, "route.counts")
    return k, E


def moe_dispatch(x, route: MoeRoute, *, stream=None):
    """Token rows ``x`` (tokens, width), bf16 or fp32, laid out group after
    group: (capacity, width) with capacity = ``moe_row_capacity(...)``; padding
    rows and rows past the last group are zeros.  ``route.offs`` are the
    groups of the result, as the jagged quantizers take them."""
    torch = _torch()
    dt = _dtype(x, 2, "x")
    T, W = x.shape
    dev = x.device
    k, E = _plan(route, T, dev)
    cap = moe_row_capacity(T, k, E, route.align)

    def call(st):
        out = torch.empty((cap, W), dtype=x.dtype, device=dev)
        code = mxq_moe_dispatch(x.data_ptr(), dt, T, W, x.stride(0), x.stride(1), route.rows.data_ptr(), k,
                                route.counts.data_ptr(), route.offs.data_ptr(), E, out.data_ptr(), cap, W, 1, st)
        _check(code, "mxq_moe_dispatch")
        return out

    return _run(x, stream, call)


def _combine(yg, route, weighted, residual, stream, name, any_layout=False):
    torch = _torch()
    dt = _dtype(yg, 2, name)
    cap, W = yg.shape
    dev = yg.device
    T = route.rows.shape[0] if route.rows is not None else 0
    k, _ = _plan(route, T, dev)
    weights = route.weights if weighted else None
    if weighted:
        _plain(weights, torch.float32, (T, k), dev, "route.weights")
    if residual is not None:
        _same(residual, yg, (T, W), "residual")

    def call(st):
        src = _unit(yg) if any_layout else yg
        y = torch.empty((T, W), dtype=yg.dtype, device=dev)
        code = mxq_moe_combine(
            src.data_ptr(), dt, cap, W, src.stride(0), src.stride(1), route.rows.data_ptr(),
            0 if weights is None else weights.data_ptr(), k, 0 if residual is None else residual.data_ptr(),
            0 if residual is None else residual.stride(0), 1 if residual is None else residual.stride(1),
            y.data_ptr(), W, 1, T, st)
        _check(code, "mxq_moe_combine")
        return y

    return _run(yg, stream, call)


def moe_dispatch_backward(grad_xg, route: MoeRoute, *, stream=None):
    """Gradient of ``moe_dispatch`` with respect to ``x``: the sum of each
    token's rows of ``grad_xg`` (capacity, width)."""
    return _combine(grad_xg, route, False, None, stream, "grad_xg", any_layout=True)


def moe_combine(yg, route: MoeRoute, *, residual=None, stream=None):
    """Expert outputs ``yg`` (capacity, width) back to the tokens:
    ``residual + sum_j weights[:, j] * yg[rows[:, j]]`` in fp32, rounded once
    to yg's type.  ``residual``: (tokens, width) of yg's type, or None."""
    return _combine(yg, route, True, residual, stream, "yg")


def moe_combine_backward(grad_y, yg, route: MoeRoute, *, stream=None):
    """Gradients of ``moe_combine``: ``(grad_yg, grad_weights)``, of yg's shape
    and type (zeros in the rows that no slot names) and (tokens, top_k) fp32.
    The residual's gradient is ``grad_y`` itself."""
    torch = _torch()
    dt = _dtype(yg, 2, "yg")
    cap, W = yg.shape
    T = grad_y.shape[0]
    _same(grad_y, yg, (T, W), "grad_y")
    k, E = _plan(route, T, yg.device)
    _plain(route.weights, torch.float32, (T, k), yg.device, "route.weights")

    def call(st):
        dy = _unit(grad_y)
        out = torch.empty((cap, W), dtype=yg.dtype, device=yg.device)
        dw = torch.empty((T, k), dtype=torch.float32, device=yg.device)
        code = mxq_moe_combine_backward(
            dy.data_ptr(), dt, T, W, dy.stride(0), dy.stride(1), yg.data_ptr(), yg.stride(0), yg.stride(1),
            route.rows.data_ptr(), route.weights.data_ptr(), k, route.counts.data_ptr(), route.offs.data_ptr(), E,
            cap, out.data_ptr(), W, 1, dw.data_ptr(), st)
        _check(code, "mxq_moe_combine_backward")
        return out, dw

    return _run(yg, stream, call)

"""The experts' products: grouped rows (``moe_dispatch``) times their expert's
weights with bias, activation, gate and residual in the product's kernel, in
bf16 with gradients and on MXFP8 operands; a whole mixture-of-experts layer for
a few tokens.

Tensor-level binding over the C ABI in ``include/mxq.h`` like the rest of the
package: shapes and types are checked, outputs allocated with torch, device
pointers and the HIP stream forwarded.  With a ``stream`` the outputs are
allocated on that stream.
"""
from __future__ import annotations

import functools

from . import MXQError, _check, _torch
from ._capi import (MXQ_ACT_GELU, MXQ_ACT_NONE, MXQ_ACT_RELU, MXQ_ACT_SILU, MXQ_BF16, MXQ_ERR_INVALID_ARG,
                    MXQ_ERR_WORKSPACE, MXQ_F32, mxq_moe_layer, mxq_moe_layer_workspace_bytes, mxq_moe_linear,
                    mxq_moe_linear_backward, mxq_moe_linear_backward_workspace_bytes, mxq_moe_linear_mx,
                    mxq_moe_linear_mx_workspace_bytes, mxq_moe_linear_workspace_bytes)
from .moe import _plain, _run, _unit

ACTIVATIONS = {"none": MXQ_ACT_NONE, "relu": MXQ_ACT_RELU, "gelu": MXQ_ACT_GELU, "silu": MXQ_ACT_SILU}


def _activation(name: str) -> int:
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}") from None


def _tensor(t, dtype, ndim: int, device, name: str) -> None:
    if t.dtype is not dtype or t.dim() != ndim or t.device != device or not t.is_cuda:
        raise TypeError(f"{name} must be a {ndim}-D {dtype} tensor on {device if device.type == 'cuda' else 'a GPU'}, "
                        f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(t, shape, device, name: str) -> None:
    _tensor(t, _torch().bfloat16, 2, device, name)
    if t.shape != shape:
        raise TypeError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _experts(w, x_width: int, offs, device, dtype, name: str):
    """w as (E, wide, width) and E, wide; the groups checked."""
    torch = _torch()
    if w.dim() == 2:
        w = w[None]
    _tensor(w, dtype, 3, device, name)
    if w.shape[2] != x_width:
        raise TypeError(f"{name} must have {x_width} columns like x, got {tuple(w.shape)}")
    if offs is not None:
        _plain(offs, torch.int32, (w.shape[0],), device, "offs")
    elif w.shape[0] != 1:
        raise TypeError(f"{name} of {w.shape[0]} experts needs offs, their group ends")
    return w


def _epilogue(rows, E, wide, device, bias, activation, gated, residual):
    """(columns of the result, the C call's arguments from bias to residual),
    checked."""
    act, gated = _activation(activation), 1 if gated else 0
    if gated and wide % 2:
        raise TypeError(f"a gated product needs an even number of weight rows, got {wide}")
    n = wide // 2 if gated else wide
    b = bs = 0
    dtype = MXQ_F32
    if bias is not None:
        torch = _torch()
        if bias.dim() == 1:
            bias = bias[None]
        if (bias.dtype not in (torch.bfloat16, torch.float32) or bias.shape != (E, wide) or bias.device != device
                or wide > 1 and bias.stride(1) != 1):
            raise TypeError(f"bias must be a bfloat16 or float32 tensor of shape {(E, wide)} and unit stride on "
                            f"{device}, got {bias.dtype} {tuple(bias.shape)} on {bias.device}")
        b, bs = bias.data_ptr(), bias.stride(0)
        if bias.dtype is torch.bfloat16:
            dtype = MXQ_BF16
    r, rs, rc = 0, 0, 1
    if residual is not None:
        _rows(residual, (rows, n), device, "residual")
        r = residual.data_ptr()
        rs, rc = residual.stride()
    return n, (b, dtype, bs, act, gated, r, rs, rc)


@functools.lru_cache(maxsize=4096)
def _need(query, *extents) -> int:
    """Workspace bytes, which the extents alone decide."""
    return query(*extents)


def _call(fn, what: str, args, query, extents, device, st) -> None:
    """The C call with the workspace that aligned operands need, most none; if
    it asks for more, with that for any operands."""
    torch = _torch()
    for aligned in (1, 0):
        n = max(_need(query, *extents, aligned), 0)
        ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None  # alive until all is launched
        code = fn(*args, _ptr(ws), n, st)
        if code != MXQ_ERR_WORKSPACE:
            break
    _check(code, what)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def moe_linear(x, w, offs=None, *, bias=None, activation: str = "none", gated: bool = False, residual=None,
               save_pre: bool = False, stream=None):
    """Rows ``x`` (rows, width) times their expert's weights ``w`` (experts,
    wide, width), both bf16: ``act(x W^T + bias) + residual``, or with
    ``gated`` ``act(first half) * second half + residual`` over wide / 2
    columns.  ``offs``: int32 group ends on the device (``route.offs``), which
    must not decrease; without them w is one expert's (2-D, or one of 3-D) and
    takes every row.
    ``activation``: "none", "relu", "gelu" or "silu"; ``bias`` (experts, wide),
    bf16 or fp32; ``residual`` (rows, n) bf16.  Returns y (rows, n) bf16, rows
    past the last group zeros; with ``save_pre`` also what the activation took
    (rows, wide), for ``moe_linear_backward``."""
    torch = _torch()
    _tensor(x, torch.bfloat16, 2, x.device, "x")
    rows, width = x.shape
    w = _experts(w, width, offs, x.device, torch.bfloat16, "w")
    E, wide, _ = w.shape
    n, epilogue = _epilogue(rows, E, wide, x.device, bias, activation, gated, residual)

    def call(st):
        y = torch.empty((rows, n), dtype=x.dtype, device=x.device)
        pre = torch.empty((rows, wide), dtype=x.dtype, device=x.device) if save_pre else None
        _call(mxq_moe_linear, "mxq_moe_linear",
              (x.data_ptr(), rows, width, *x.stride(), w.data_ptr(), E, wide, *w.stride(), _ptr(offs), *epilogue,
               y.data_ptr(), n or 1, 1, _ptr(pre), wide or 1, 1),
              mxq_moe_linear_workspace_bytes, (rows, width, E, wide), x.device, st)
        return (y, pre) if save_pre else y

    return _run(x, stream, call)


def moe_linear_backward(grad_y, x, w, offs=None, *, pre=None, activation: str = "none", gated: bool = False,
                        bias: bool = False, need_x: bool = True, need_w: bool = True, stream=None):
    """Gradients of ``moe_linear``: ``(grad_x, grad_w, grad_bias)``, bf16, bf16
    and fp32 (experts, wide), None for what is not asked for.  ``pre`` is what
    the forward call saved, needed with an activation or a gate.  The
    residual's gradient is ``grad_y`` itself."""
    torch = _torch()
    _tensor(x, torch.bfloat16, 2, x.device, "x")
    rows, width = x.shape
    w = _experts(w, width, offs, x.device, torch.bfloat16, "w")
    E, wide, _ = w.shape
    act, gated = _activation(activation), 1 if gated else 0
    if gated and wide % 2:
        raise TypeError(f"a gated product needs an even number of weight rows, got {wide}")
    _rows(grad_y, (rows, wide // 2 if gated else wide), x.device, "grad_y")
    saved = act != MXQ_ACT_NONE or gated
    if saved:
        if pre is None:
            raise TypeError("an activation or a gate needs pre, what moe_linear(..., save_pre=True) returned")
        _rows(pre, (rows, wide), x.device, "pre")

    def call(st):
        g = _unit(grad_y)
        dx = torch.empty((rows, width), dtype=x.dtype, device=x.device) if need_x else None
        dw = torch.empty((E, wide, width), dtype=x.dtype, device=x.device) if need_w else None
        db = torch.empty((E, wide), dtype=torch.float32, device=x.device) if bias else None
        _call(mxq_moe_linear_backward, "mxq_moe_linear_backward",
              (g.data_ptr(), *g.stride(), x.data_ptr(), rows, width, *x.stride(), w.data_ptr(), E, wide, *w.stride(),
               _ptr(offs), pre.data_ptr() if saved else 0, pre.stride(0) if saved else 0, pre.stride(1) if saved else 1,
               act, gated, _ptr(dx), width, 1, _ptr(dw), wide * width, width, 1, _ptr(db)),
              mxq_moe_linear_backward_workspace_bytes, (rows, width, E, wide, act, gated, 1 if bias else 0), x.device, st)
        return dx, dw, db

    return _run(x, stream, call)


def moe_linear_mx(x, x_scales, w, w_scales, offs=None, *, bias=None, activation: str = "none", gated: bool = False,
                  residual=None, save_pre: bool = False, stream=None):
    """``moe_linear`` on MXFP8 operands with blocks along ``width``: ``x``
    (rows, width) e4m3 with ``x_scales`` (rows, width / 32) uint8, as
    ``quantize_mx_rowwise`` returns them, ``w`` (experts, wide, width) with
    ``w_scales`` (experts, wide, width / 32).  Weights quantized along N
    (``quantize_mx_3d_colwise``) are the operands of the product with their
    transposes, which is the gradient with respect to x:
    ``moe_linear_mx(*quantize_mx_rowwise(grad_z), q.transpose(1, 2),
    scales.transpose(1, 2), offs)``."""
    torch = _torch()
    f8 = torch.float8_e4m3fn
    _tensor(x, f8, 2, x.device, "x")
    rows, width = x.shape
    w = _experts(w, width, offs, x.device, f8, "w")
    E, wide, _ = w.shape
    if w_scales.dim() == 2:
        w_scales = w_scales[None]
    for t, shape, name in ((x_scales, (rows, width // 32), "x_scales"), (w_scales, (E, wide, width // 32), "w_scales")):
        _tensor(t, torch.uint8, len(shape), x.device, name)
        if t.shape != shape or width % 32:
            raise TypeError(f"{name} must have shape {shape} for blocks of 32 of {width}, got {tuple(t.shape)}")
    n, epilogue = _epilogue(rows, E, wide, x.device, bias, activation, gated, residual)

    def call(st):
        y = torch.empty((rows, n), dtype=torch.bfloat16, device=x.device)
        pre = torch.empty((rows, wide), dtype=torch.bfloat16, device=x.device) if save_pre else None
        _call(mxq_moe_linear_mx, "mxq_moe_linear_mx",
              (x.data_ptr(), rows, width, *x.stride(), x_scales.data_ptr(), *x_scales.stride(), w.data_ptr(), E, wide,
               *w.stride(), w_scales.data_ptr(), *w_scales.stride(), _ptr(offs), *epilogue, y.data_ptr(), n or 1, 1,
               _ptr(pre), wide or 1, 1), mxq_moe_linear_mx_workspace_bytes, (rows, width, E, wide), x.device, st)
        return (y, pre) if save_pre else y

    return _run(x, stream, call)


# ---------------------------------------------------------------- a layer for a few tokens

def _weights(w, shape, device, name: str):
    """(tensor, scales or None) of expert weights: bf16, or MXFP8 as a pair."""
    torch = _torch()
    if not isinstance(w, (tuple, list)):
        _tensor(w, torch.bfloat16, 3, device, name)
        q, scales = w, None
    else:
        q, scales = w
        _tensor(q, torch.float8_e4m3fn, 3, device, name)
        _tensor(scales, torch.uint8, 3, device, f"{name}'s scales")
        blocks = shape[:2] + (shape[2] // 32,)
        if scales.shape != blocks or shape[2] % 32:
            raise TypeError(f"{name}'s scales must have shape {blocks} for blocks of 32 of {shape[2]}, got {tuple(scales.shape)}")
    if q.shape != shape:
        raise TypeError(f"{name} must have shape {shape}, got {tuple(q.shape)}")
    return q, scales


def _layer_bias(bias, shape, device, name: str):
    torch = _torch()
    if bias is None:
        return 0, 0, MXQ_F32
    if (bias.dtype not in (torch.bfloat16, torch.float32) or bias.shape != shape or bias.device != device
            or shape[1] > 1 and bias.stride(1) != 1):
        raise TypeError(f"{name} must be a bfloat16 or float32 tensor of shape {shape} and unit stride on {device}, got "
                        f"{bias.dtype} {tuple(bias.shape)} on {bias.device}")
    return bias.data_ptr(), bias.stride(0), MXQ_BF16 if bias.dtype == torch.bfloat16 else MXQ_F32


def moe_layer_workspace(tokens: int, width: int, hidden: int, num_experts: int, top_k: int, device=None):
    """A workspace for ``moe_layer(..., workspace=ws)`` of this extent; it can
    be reused by calls that do not overlap in time."""
    need = mxq_moe_layer_workspace_bytes(tokens, width, hidden, num_experts, top_k)
    if need < 0:
        raise MXQError(MXQ_ERR_INVALID_ARG, "mxq_moe_layer_workspace_bytes")
    return _torch().empty(max(need, 16), dtype=_torch().uint8, device=device or "cuda")


def moe_layer(x, logits, up, down, top_k: int, *, activation: str = "silu", gated: bool = True, bias_up=None,
              bias_down=None, token_mask=None, renormalize: bool = True, residual=None, workspace=None, stream=None):
    """A whole mixture-of-experts layer for up to 64 tokens ``x`` (tokens,
    width) bf16: the ``top_k`` experts of their router ``logits`` (tokens,
    experts), bf16 or fp32, as ``moe_route`` chooses and weighs them; ``up``
    (experts, hidden or with ``gated`` 2 hidden, width), the activation,
    ``down`` (experts, width, hidden), the weighted sum and the ``residual``.
    Weights are bf16 tensors, or pairs ``(q, scales)`` of MXFP8 blocks along
    their last dim.  Every active expert's weights are read once.  More tokens:
    ``moe_route``, ``moe_dispatch``, ``moe_linear``, ``moe_combine``."""
    torch = _torch()
    _tensor(x, torch.bfloat16, 2, x.device, "x")
    T, D = x.shape
    dev = x.device
    if logits.dim() != 2 or logits.dtype not in (torch.bfloat16, torch.float32) or logits.device != dev or logits.shape[0] != T:
        raise TypeError(f"logits must be a bfloat16 or float32 tensor of {T} rows on {dev}, got {logits.dtype} "
                        f"{tuple(logits.shape)} on {logits.device}")
    E = logits.shape[1]
    act = _activation(activation)
    q = down[0] if isinstance(down, (tuple, list)) else down
    H = q.shape[-1]
    wide = 2 * H if gated else H
    (uq, us), (dq, ds) = _weights(up, (E, wide, D), dev, "up"), _weights(down, (E, D, H), dev, "down")
    if (us is None) != (ds is None):
        raise TypeError("up and down must have the same format")
    bu, bus, bdt = _layer_bias(bias_up, (E, wide), dev, "bias_up")
    bd, bds, bdt2 = _layer_bias(bias_down, (E, D), dev, "bias_down")
    if bias_up is not None and bias_down is not None and bdt != bdt2:
        raise TypeError("bias_up and bias_down must have the same type")
    if residual is not None:
        _rows(residual, (T, D), dev, "residual")
    if token_mask is not None:
        if token_mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"token_mask must be a bool or uint8 tensor, got {token_mask.dtype}")
        _plain(token_mask, token_mask.dtype, (T,), dev, "token_mask")
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise TypeError("workspace must be a contiguous CUDA tensor on x's device")
    k = int(top_k)
    need = mxq_moe_layer_workspace_bytes(T, D, H, E, k)
    if need < 0:
        raise MXQError(MXQ_ERR_INVALID_ARG, "mxq_moe_layer")

    def call(st):
        y = torch.empty((T, D), dtype=x.dtype, device=dev)
        ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8, device=dev)
        none = (0, 0, 0)
        code = mxq_moe_layer(
            x.data_ptr(), T, D, *x.stride(), logits.data_ptr(), MXQ_BF16 if logits.dtype == torch.bfloat16 else MXQ_F32, E,
            *logits.stride(), _ptr(token_mask), k, int(bool(renormalize)), H, int(us is not None),
            uq.data_ptr(), _ptr(us), *uq.stride(), *(none if us is None else us.stride()), bu,
            dq.data_ptr(), _ptr(ds), *dq.stride(), *(none if ds is None else ds.stride()), bd,
            bdt if bias_up is not None else bdt2, bus, bds, act, int(bool(gated)), _ptr(residual),
            0 if residual is None else residual.stride(0), 1 if residual is None else residual.stride(1), y.data_ptr(), D, 1,
            ws.data_ptr(), ws.numel() * ws.element_size(), st)
        _check(code, "mxq_moe_layer")
        return y

    return _run(x, stream, call)

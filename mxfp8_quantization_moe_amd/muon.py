"""Newton-Schulz orthogonalisation of weight updates: the step the Muon
optimiser applies to each expert's momentum before it is subtracted from the
weights (and those quantized again)."""
from __future__ import annotations

from . import MXQError, _check, _torch
from ._capi import (MXQ_BF16, MXQ_ERR_INVALID_ARG, MXQ_F32, mxq_muon_orthogonalize, mxq_muon_workspace_bytes)
from .moe import _run

MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _need(count: int, rows: int, cols: int) -> int:
    n = mxq_muon_workspace_bytes(count, rows, cols)
    if n < 0:
        raise MXQError(MXQ_ERR_INVALID_ARG, "mxq_muon_workspace_bytes")
    return n


def muon_workspace(count: int, rows: int, cols: int, device=None):
    """A workspace for ``muon_orthogonalize(..., workspace=ws)`` on matrices
    of this extent; it can be reused by calls that do not overlap in time."""
    torch = _torch()
    return torch.empty(max(_need(count, rows, cols), 16), dtype=torch.uint8, device=device or "cuda")


def muon_orthogonalize(g, *, steps: int = 5, coefficients=MUON_COEFFICIENTS, eps: float = 1e-7, scale: float = 1.0,
                       workspace=None, stream=None):
    """``scale`` times the orthogonalised update of every matrix in ``g``:
    (rows, cols) or (count, rows, cols), bf16 or fp32, each matrix row- or
    column-major.  Returns a contiguous bf16 tensor of g's shape (see
    mxq_muon_orthogonalize in ``include/mxq.h`` for the formula and the
    numerics).  Without a ``workspace`` (``muon_workspace``) one is allocated
    for the call."""
    torch = _torch()
    if g.dim() not in (2, 3) or g.dtype not in (torch.bfloat16, torch.float32) or not g.is_cuda:
        raise TypeError(f"g must be a 2-D or 3-D bfloat16 or float32 CUDA tensor, got {g.dtype} {tuple(g.shape)} on "
                        f"{g.device}")
    count = g.shape[0] if g.dim() == 3 else 1
    rows, cols = g.shape[-2:]
    a, b, c = (float(v) for v in coefficients)
    if workspace is not None and (not workspace.is_cuda or workspace.device != g.device or not workspace.is_contiguous()):
        raise TypeError("workspace must be a contiguous CUDA tensor on g's device")
    need = _need(count, rows, cols)

    def call(st):
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
        ws = workspace if workspace is not None else torch.empty(max(need, 16), dtype=torch.uint8, device=g.device)
        code = mxq_muon_orthogonalize(
            g.data_ptr(), MXQ_BF16 if g.dtype == torch.bfloat16 else MXQ_F32, count, rows, cols,
            g.stride(0) if g.dim() == 3 else 0, g.stride(-2), g.stride(-1), out.data_ptr(), rows * cols, cols, 1,
            int(steps), a, b, c, float(eps), float(scale), ws.data_ptr(), ws.numel() * ws.element_size(), st)
        _check(code, "mxq_muon_orthogonalize")
        return out

    return _run(g, stream, call)

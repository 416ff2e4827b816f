"""Orthogonalised updates: what an optimiser steps along, made of the weight gradients that
the loss and the blocks before it return.  Through ``slm_orthogonalize``."""

from __future__ import annotations

import torch

from . import _lib
from .loss import _ptr, _stream
from .norms import _DTYPE, _overlap

#: Five steps of it move singular values from [0.002, 1] into [0.68, 1.21], from [0.01, 1] into [0.68, 1.14].
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize_workspace_bytes(batch, m, n):
    """Bytes of workspace for a stack of ``batch`` [m, n] matrices (0: sizes not supported)."""
    return int(_lib.slm_orthogonalize_workspace_bytes(batch, m, n))


def _steps(coefficients, steps):
    """One (a, b, c) per step, from one triple for all steps or one each."""
    try:
        n = int(steps)
    except (TypeError, ValueError):
        n = 0
    if n < 1 or n > 64 or n != steps:
        raise ValueError(f"steps must be a whole number from 1 to 64, not {steps}")
    try:
        rows = [tuple(float(v) for v in c) for c in coefficients]
    except TypeError:
        rows = [tuple(float(v) for v in coefficients)] * n
    if len(rows) != n or any(len(r) != 3 for r in rows):
        raise ValueError("coefficients must be one (a, b, c) or one for each step")
    return rows


def orthogonalize(grad, momentum=None, beta=0.95, nesterov=True, steps=5,
                  coefficients=COEFFICIENTS, eps=1e-7, out=None, workspace=None):
    """Orthogonalised update of one matrix [m, n] or a stack [batch, m, n]::

        momentum <- beta momentum + (1 - beta) grad             (in place, if given)
        u = beta momentum + (1 - beta) grad  (nesterov), momentum, or grad without one
        X = u / (||u||_F + eps)
        steps times:  A = X X^T,  X <- a X + (b A + c A^2) X    (X^T X on the right when m > n)

    ``grad`` is a bf16, fp16 or fp32 CUDA tensor with adjacent columns (rows and matrices may
    be strided) and is not written; ``momentum`` is a contiguous float32 tensor of its shape;
    ``coefficients`` is one (a, b, c), or a sequence of one per step, within the range that
    ``slm_orthogonalize`` documents.  Returns X as a contiguous bf16 tensor of grad's shape
    (``out`` if given).  ``workspace`` may be a uint8 tensor of
    ``orthogonalize_workspace_bytes``.  ``device_status()`` tells of waits that ran out: what the
    call returned is then undefined, and ``momentum`` may have been advanced."""
    if not isinstance(grad, torch.Tensor) or not grad.is_cuda or grad.dim() not in (2, 3):
        raise ValueError("grad must be a 2-D or 3-D CUDA tensor")
    if grad.dtype not in _DTYPE:
        raise ValueError(f"grad must be bf16, fp16 or fp32, not {grad.dtype}")
    dev = grad.device
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"grad is on {dev}, not on the current CUDA device")
    shape = tuple(grad.shape)
    g = grad if grad.dim() == 3 else grad.unsqueeze(0)
    batch, m, n = g.shape
    ld = g.stride(1) if m > 1 else n
    stack = g.stride(0) if batch > 1 else 0
    if (n > 1 and g.stride(2) != 1) or ld < n or (batch > 1 and stack < (m - 1) * ld + n):
        raise ValueError(f"grad must have adjacent columns, and rows and matrices that do not "
                         f"overlap; its strides are {grad.stride()}")
    rows = _steps(coefficients, steps)
    if not 0.0 <= beta <= 1.0:
        raise ValueError("beta must be within [0, 1]")
    if not eps >= 2.0 ** -126:
        raise ValueError("eps must be positive, and normal in float32")
    for name, t, dtype in (("momentum", momentum, torch.float32), ("out", out, torch.bfloat16)):
        if t is None:
            continue
        if (not t.is_cuda or t.device != dev or t.dtype != dtype or tuple(t.shape) != shape
                or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {dev}")
    for a, b, what in ((out, grad, "out overlaps grad"), (out, momentum, "out overlaps momentum"),
                       (momentum, grad, "momentum overlaps grad")):
        if _overlap(a, b):
            raise ValueError(what)
    need = orthogonalize_workspace_bytes(batch, m, n)
    if need == 0:
        raise ValueError(f"a stack of shape {shape} is too large")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif (workspace.dtype != torch.uint8 or workspace.device != dev
          or not workspace.is_contiguous() or workspace.numel() < need):
        raise ValueError(f"workspace must be a contiguous uint8 tensor of {need} bytes on {dev}")
    written = [t for t in (momentum, out) if t is not None]
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    st = _lib.slm_orthogonalize(_DTYPE[grad.dtype], _ptr(grad), ld, stack, batch, m, n,
                                _ptr(momentum), beta, nesterov, rows, eps, _ptr(out),
                                _ptr(workspace), workspace.numel(), _stream())
    _lib.check(st, "slm_orthogonalize")
    for t in written:   # in place: autograd is to know
        torch.autograd.graph.increment_version(t)
    return out

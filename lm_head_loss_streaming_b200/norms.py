"""Norms before and after a draft block, fused with its gate and its residual scale.

``block_norm`` makes, in one pass over the rows, the residual stream after a block and the
normalised hidden states that the next block or ``streaming_lm_head_loss`` reads; its
backward takes the gradient that the loss returns for them.  Through ``slm_block_norm_fwd``
and ``slm_block_norm_bwd``.
"""

from __future__ import annotations

import functools
from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .loss import _ptr

_DTYPE = {torch.bfloat16: _lib.SLM_BF16, torch.float16: _lib.SLM_F16,
          torch.float32: _lib.SLM_F32}


@dataclass
class BlockNormResult:
    residual: torch.Tensor            # [N, d], the inputs' type; x itself without y
    hidden: torch.Tensor | None       # [N, d]; None without w_pre
    stats: torch.Tensor               # float32 [2, N]: 1 / sqrt(mean + eps) of the norms of y and
                                      # of the residual (each written if there is that norm)
    residual_scale: float
    block_scale: float
    weight_offset: float


@dataclass
class BlockNormGrads:
    dx: torch.Tensor                  # [N, d], the inputs' type
    dy: torch.Tensor | None           # [N, d]
    dgate: torch.Tensor | None        # the gate's shape and type
    dw_pre: torch.Tensor | None       # float32 [d]
    dw_post: torch.Tensor | None      # float32 [d]


def _current(x):
    """(current device, raw stream handle of its current stream), once x is seen to be on a GPU."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("the inputs must be CUDA tensors")
    dev = torch._C._cuda_getDevice()
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _check_rows(name, t, N, d, dtype, dev):
    """Rows [N, d] on the current device, elements of a row adjacent, rows apart; returns the
    distance between rows."""
    if t.dtype is not dtype or t.shape != (N, d) or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {(N, d)} on the current CUDA "
                         f"device")
    ld, step = t.stride()
    if N <= 1:
        ld = d
    if ld < d or (step != 1 and d > 1):
        raise ValueError(f"{name} must have adjacent channels and rows that do not overlap; its "
                         f"strides are {t.stride()}")
    return ld


def _check_weight(name, t, d, dtype, dev):
    if t.shape != (d,) or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape ({d},) on the "
                         f"current CUDA device (both weights of the inputs' type, or float32)")


def _check_block(x, y, w_pre, w_post, gate, dev):
    """Raises ValueError unless the inputs are what the kernels are told; returns
    (N, d, dtype id, row strides of x and y, weight dtype id, gate dtype id, gate rows)."""
    dtype = x.dtype
    dt = _DTYPE.get(dtype)
    if dt is None or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16, fp16 or fp32 CUDA tensor")
    N, d = x.shape
    if d < 1:
        raise ValueError("x has rows of no channels")
    ldx = ldy = _check_rows("x", x, N, d, dtype, dev)
    if y is not None:
        ldy = _check_rows("y", y, N, d, dtype, dev)
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate apply to y, which is missing")
    elif w_pre is None:
        raise ValueError("nothing to do: neither y nor w_pre is given")
    wt = gt = dt
    rows = 0
    if w_pre is not None or w_post is not None:
        w_dtype = (w_pre if w_pre is not None else w_post).dtype
        if w_dtype is not dtype:
            if w_dtype is not torch.float32:
                raise ValueError(f"the weights must be {dtype} or float32")
            wt = _lib.SLM_F32
        if w_pre is not None:
            _check_weight("w_pre", w_pre, d, w_dtype, dev)
        if w_post is not None:
            _check_weight("w_post", w_post, d, w_dtype, dev)
    if gate is not None:
        shape = gate.shape
        if (gate.get_device() != dev or len(shape) not in (1, 2) or shape[-1] != d
                or not gate.is_contiguous() or gate.dtype not in (dtype, torch.float32)):
            raise ValueError(f"gate must be a contiguous tensor of shape ({d},) or (rows, {d}) on "
                             f"the current CUDA device, of {dtype} or float32")
        rows = 1 if len(shape) == 1 else shape[0]
        if N > 0 and (rows == 0 or N % rows != 0):
            raise ValueError(f"gate has {rows} rows; they must divide the {N} rows of x")
        if gate.dtype is not dtype:
            gt = _lib.SLM_F32
    return N, d, dt, ldx, ldy, wt, gt, rows


@functools.lru_cache(maxsize=256)
def _workspace_bytes(N, d, rows):
    return _lib.slm_block_norm_workspace_bytes(N, d, rows)


def _overlap(a, b):
    """Whether two tensors' address ranges meet."""
    if a is None or b is None or a.numel() == 0 or b.numel() == 0:
        return False

    def span(t):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()

    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


def _check_outputs(outs, ins, may_be=None):
    """Caller-provided outputs overlap neither an input nor each other (``may_be``: the pair
    (output, input) that may be the same tensor)."""
    for i, (name, t) in enumerate(outs):
        for other, u in list(ins) + outs[:i]:
            if _overlap(t, u) and not (may_be == (name, other) and t.data_ptr() == u.data_ptr()
                                       and u.is_contiguous()):
                raise ValueError(f"{name} overlaps {other}")


def block_norm_fwd(x, y=None, w_pre=None, w_post=None, gate=None, residual_scale=1.0,
                   block_scale=1.0, eps=1e-6, weight_offset=0.0, residual=None, hidden=None
                   ) -> BlockNormResult:
    """Residual stream and normalised hidden states after a block, through
    ``slm_block_norm_fwd``::

        v        = norm(y) * (w_post + weight_offset)      (v = y without w_post)
        residual = residual_scale * x + block_scale * gate * v
        hidden   = norm(residual) * (w_pre + weight_offset)
        norm(t)  = t / sqrt(mean(t^2) + eps)

    ``x`` (the stream) and ``y`` (the block's output) are [N, d] bf16, fp16 or fp32 CUDA
    tensors with adjacent channels; rows may be strided.  ``w_pre`` and ``w_post`` are [d],
    ``gate`` [d] or [G, d] with G dividing N (each gate row covers N / G rows in a row: a gate
    per channel, per sequence or per token), of the inputs' type or float32.  Without ``y``
    only ``hidden`` is made, of ``x`` (residual_scale must be 1); without ``w_pre`` only the
    residual.  ``residual`` and ``hidden`` may be preallocated contiguous outputs;
    ``residual`` may be ``x`` itself, which is then updated in place (a backward needs the old
    ``x``).

    Rows may begin anywhere, but inputs that do not begin on 16-byte boundaries, beside outputs
    that do (as all outputs made here do), run four times slower, in the backward ten times."""
    dev, stream = _current(x)
    N, d, dt, ldx, ldy, wt, gt, rows = _check_block(x, y, w_pre, w_post, gate, dev)
    if y is None:
        if residual_scale != 1.0:
            raise ValueError("residual_scale needs y: without a block the stream is x itself")
        if residual is not None:
            raise ValueError("residual is an output of the block's add: there is none without y")
    if w_pre is None and hidden is not None:
        raise ValueError("hidden is made by the norm before the next block: there is no w_pre")
    if not eps >= 2.0 ** -126:
        raise ValueError("eps must be positive, and normal in float32")
    given = []
    if residual is not None or hidden is not None:
        given = [(n, t) for n, t in (("residual", residual), ("hidden", hidden)) if t is not None]
        for name, t in given:
            _check_rows(name, t, N, d, x.dtype, dev)
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        _check_outputs(given, [("x", x), ("y", y), ("w_pre", w_pre), ("w_post", w_post),
                               ("gate", gate)], ("residual", "x"))
    if y is not None and residual is None:
        residual = torch.empty_like(x) if ldx == d else x.new_empty((N, d))
    if w_pre is not None and hidden is None:
        hidden = torch.empty_like(x) if ldx == d else x.new_empty((N, d))
    stats = x.new_empty((2, N), dtype=torch.float32)
    at = stats.data_ptr()
    st = _lib.slm_block_norm_fwd(dt, x.data_ptr(), ldx, _ptr(y), ldy, _ptr(w_post), _ptr(w_pre),
                                 wt, _ptr(gate), gt, rows, N, d, residual_scale, block_scale, eps,
                                 weight_offset, _ptr(residual), _ptr(hidden), at, at + 4 * N,
                                 stream)
    if st:
        raise _lib.SLMError(st, "slm_block_norm_fwd")
    for _, t in given:   # written in place: autograd is to know
        torch.autograd.graph.increment_version(t)
    return BlockNormResult(x if y is None else residual, hidden, stats, residual_scale,
                           block_scale, weight_offset)


def block_norm_bwd(fwd: BlockNormResult, x, y=None, w_pre=None, w_post=None, gate=None,
                   d_residual=None, d_hidden=None, workspace=None) -> BlockNormGrads:
    """Gradients of ``block_norm_fwd`` for the same inputs, through ``slm_block_norm_bwd``.

    ``d_residual`` and ``d_hidden`` are the gradients of its two outputs (``d_residual`` may
    be None: zero).  ``dx`` and ``dy`` have the inputs' type, ``dgate`` the gate's shape and
    type (summed over the rows that share a gate row), the weights' gradients are float32.
    The sums run in a fixed order.  ``workspace`` may hold a uint8 tensor of
    ``slm_block_norm_workspace_bytes``.  ``device_status()`` tells of waits that ran out."""
    dev, stream = _current(x)
    N, d, dt, ldx, ldy, wt, gt, rows = _check_block(x, y, w_pre, w_post, gate, dev)
    if (w_pre is None) != (d_hidden is None) or (d_hidden is None and d_residual is None):
        raise ValueError("d_hidden is the gradient of hidden, made with w_pre: give both or "
                         "neither, and at least one gradient")
    ld_dr = ld_dh = d
    if d_residual is not None:
        ld_dr = _check_rows("d_residual", d_residual, N, d, x.dtype, dev)
    if d_hidden is not None:
        ld_dh = _check_rows("d_hidden", d_hidden, N, d, x.dtype, dev)
    stats = fwd.stats
    if (stats.shape != (2, N) or stats.get_device() != dev or stats.dtype is not torch.float32
            or not stats.is_contiguous()):
        raise ValueError("fwd does not come from a forward over these inputs")
    device = x.device
    need = _workspace_bytes(N, d, rows if N > 0 else 0)
    if workspace is None:
        workspace = x.new_empty(need, dtype=torch.uint8)
    elif (workspace.dtype != torch.uint8 or workspace.device != device
          or not workspace.is_contiguous() or workspace.numel() < need):
        raise ValueError(f"workspace must be a contiguous uint8 tensor of {need} bytes on {device}")
    g = BlockNormGrads(
        x.new_empty((N, d)), None if y is None else x.new_empty((N, d)),
        None if gate is None else torch.empty_like(gate) if N > 0 else torch.zeros_like(gate),
        None if w_pre is None else x.new_empty(d, dtype=torch.float32),
        None if w_post is None else x.new_empty(d, dtype=torch.float32))
    at = stats.data_ptr()
    st = _lib.slm_block_norm_bwd(dt, x.data_ptr(), ldx, _ptr(y), ldy, _ptr(w_post), _ptr(w_pre),
                                 wt, _ptr(gate), gt, rows, _ptr(d_residual), ld_dr,
                                 _ptr(d_hidden), ld_dh, at, at + 4 * N, N, d, fwd.residual_scale,
                                 fwd.block_scale, fwd.weight_offset, g.dx.data_ptr(), _ptr(g.dy),
                                 _ptr(g.dgate), _ptr(g.dw_post), _ptr(g.dw_pre),
                                 workspace.data_ptr(), workspace.numel(), stream)
    if st:
        raise _lib.SLMError(st, "slm_block_norm_bwd")
    return g


class BlockNorm(torch.autograd.Function):
    """(residual, hidden) of ``block_norm_fwd`` with its gradients."""

    @staticmethod
    def forward(ctx, x, y, w_pre, w_post, gate, residual_scale, block_scale, eps, weight_offset):
        fwd = block_norm_fwd(x, y, w_pre, w_post, gate, residual_scale, block_scale, eps,
                             weight_offset)
        ctx.save_for_backward(x, y, w_pre, w_post, gate, fwd.stats)
        ctx.scales = (fwd.residual_scale, fwd.block_scale, fwd.weight_offset)
        ctx.set_materialize_grads(False)
        return None if y is None else fwd.residual, fwd.hidden

    @staticmethod
    @once_differentiable
    def backward(ctx, d_residual, d_hidden):
        x, y, w_pre, w_post, gate, stats = ctx.saved_tensors
        if d_residual is None and d_hidden is None:
            return (None,) * 9
        if w_pre is not None and d_hidden is None:   # hidden was not used
            d_hidden = torch.zeros_like(x, memory_format=torch.contiguous_format)
        d_residual, d_hidden = (
            None if t is None else t if t.stride(-1) == 1 and t.stride(0) >= t.shape[1]
            else t.contiguous() for t in (d_residual, d_hidden))
        fwd = BlockNormResult(None, None, stats, *ctx.scales)
        g = block_norm_bwd(fwd, x, y, w_pre, w_post, gate, d_residual, d_hidden)
        return (g.dx, g.dy, None if w_pre is None else g.dw_pre.to(w_pre.dtype),
                None if w_post is None else g.dw_post.to(w_post.dtype), g.dgate,
                None, None, None, None)


def block_norm(x, y=None, w_pre=None, w_post=None, gate=None, residual_scale=1.0,
               block_scale=1.0, eps=1e-6, weight_offset=0.0):
    """(residual, hidden) as ``block_norm_fwd`` makes them, differentiable with respect to
    every tensor argument.  Without ``y`` the residual is ``x``; without ``w_pre`` hidden is
    None."""
    residual, hidden = BlockNorm.apply(x, y, w_pre, w_post, gate, residual_scale, block_scale,
                                       eps, weight_offset)
    return (x if y is None else residual), hidden

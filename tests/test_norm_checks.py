"""Refusals of the block norm, before anything is launched: by the Python wrappers (wrong
device, type, layout or extent) and by the C ABI (sizes, types, pointers)."""

import ctypes

import pytest
import torch

from lm_head_loss_streaming_b200 import _lib, block_norm, block_norm_bwd, block_norm_fwd
from lm_head_loss_streaming_b200.norms import BlockNormResult, _overlap

A = 1 << 20   # an aligned address that is never read on these paths


def _fwd(**kw):
    a = dict(dtype=_lib.SLM_BF16, x=A, ldx=64, y=2 * A, ldy=64, w_post=3 * A, w_pre=4 * A,
             w_dtype=_lib.SLM_BF16, gate=5 * A, gate_dtype=_lib.SLM_BF16, gate_rows=2, N=8, d=64,
             rs=1.0, bs=1.0, eps=1e-6, off=0.0, residual=6 * A, hidden=7 * A, rstd_post=8 * A,
             rstd_pre=9 * A, stream=None)
    a.update(kw)
    return _lib.slm_block_norm_fwd(*a.values())


def _bwd(**kw):
    a = dict(dtype=_lib.SLM_BF16, x=A, ldx=64, y=2 * A, ldy=64, w_post=3 * A, w_pre=4 * A,
             w_dtype=_lib.SLM_BF16, gate=5 * A, gate_dtype=_lib.SLM_BF16, gate_rows=2, dr=6 * A,
             ld_dr=64, dh=7 * A, ld_dh=64, rstd_post=8 * A, rstd_pre=9 * A, N=8, d=64, rs=1.0,
             bs=1.0, off=0.0, dx=10 * A, dy=11 * A, dgate=12 * A, dw_post=13 * A, dw_pre=14 * A,
             ws=16 * A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return _lib.slm_block_norm_bwd(*a.values())


NAN, INF = float("nan"), float("inf")
COMMON = [
    (dict(dtype=3), 4), (dict(dtype=-1), 4), (dict(w_dtype=_lib.SLM_F16), 4),
    (dict(gate_dtype=_lib.SLM_F16), 4), (dict(N=-1), 2), (dict(d=0), 2), (dict(N=1 << 31), 2),
    (dict(d=1 << 31), 2), (dict(ldx=63), 2), (dict(ldy=63), 2), (dict(gate_rows=3), 2),
    (dict(gate_rows=0), 2), (dict(gate_rows=16), 2), (dict(rs=NAN), 2), (dict(bs=INF), 2),
    (dict(off=NAN), 2), (dict(x=None), 1), (dict(y=None), 1), (dict(x=A + 1), 3),
    (dict(w_pre=4 * A + 1), 3), (dict(gate=5 * A + 1), 3),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(eps=0.0), 2), (dict(eps=-1.0), 2), (dict(eps=NAN), 2), (dict(hidden=None), 1),
    (dict(residual=A, ldx=128), 2), (dict(residual=6 * A + 1), 3), (dict(rstd_pre=9 * A + 2), 3),
    (dict(w_pre=None, residual=None), 1)])
def test_forward_refusals(kw, status):
    assert _fwd(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(dh=None), 1), (dict(w_pre=None, dw_pre=None), 1), (dict(dx=None), 1), (dict(dy=None), 1),
    (dict(dgate=None), 1), (dict(dw_pre=None), 1), (dict(dw_post=None), 1),
    (dict(rstd_post=None), 1), (dict(rstd_pre=None), 1), (dict(ws=None), 1), (dict(ld_dr=63), 2),
    (dict(ld_dh=1), 2), (dict(ws_bytes=16), 5), (dict(ws=16 * A + 16), 5), (dict(dx=A + 1), 3),
    (dict(dw_pre=14 * A + 2), 3)])
def test_backward_refusals(kw, status):
    assert _bwd(**kw) == status


def test_nothing_to_do_is_fine_without_rows():
    assert _fwd(N=0, x=None, y=None) == _lib.SLM_OK


def test_workspace_sizes():
    assert _lib.slm_block_norm_workspace_bytes(10, 0, 0) == 0
    assert _lib.slm_block_norm_workspace_bytes(10, 8, 3) == 0
    assert _lib.slm_block_norm_workspace_bytes(-1, 8, 0) == 0
    # Partials of a bounded number of row blocks, whatever the rows and the groups.
    for gate_rows in (0, 1, 2, 4096, 65536):
        ws = _lib.slm_block_norm_workspace_bytes(65536, 4096, gate_rows)
        assert 0 < ws <= 65536 * 4 + 3 * 592 * 4096 * 4 + 4096


def test_cpu_tensors_and_missing_parts_are_refused():
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(16, dtype=torch.bfloat16)
    for kw in (dict(x=x, y=x, w_pre=w), dict(x=x, w_pre=w), dict(x=x[0], w_pre=w),
               dict(x=x.double(), w_pre=w)):
        with pytest.raises(ValueError):
            block_norm_fwd(**kw)
        with pytest.raises(ValueError):
            block_norm(**kw)


def test_overlap_of_address_ranges():
    t = torch.zeros(10, 8)
    assert _overlap(t, t[3:4]) and _overlap(t[:, :4], t[:, 4:])
    assert not _overlap(t[:5], t[5:]) and not _overlap(t, None) and not _overlap(t[:0], t)


@pytest.mark.gpu
def test_wrapper_refusals():
    x = torch.zeros(6, 32, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(32, dtype=torch.bfloat16, device="cuda")
    ok = dict(x=x, y=x.clone(), w_pre=w, w_post=w, gate=w)
    f = block_norm_fwd(**ok)
    bad = [dict(y=x[:5]), dict(y=x.float()), dict(y=None), dict(w_pre=w[:31]),
           dict(w_pre=w.float()), dict(w_post=w.half(), w_pre=w.half()), dict(gate=x[:4]),
           dict(gate=x.t()[:6]), dict(gate=w.half()), dict(x=x.t().contiguous().t()),
           dict(x=x[:1].expand(6, 32)), dict(eps=0.0), dict(eps=-1.0), dict(w_pre=w.cpu()),
           dict(residual=x[:5]), dict(residual=ok["y"]), dict(hidden=x),
           dict(hidden=torch.empty(6, 64, dtype=torch.bfloat16, device="cuda")[:, :32]),
           dict(residual=x.float())]
    for kw in bad:
        with pytest.raises(ValueError):
            block_norm_fwd(**{**ok, **kw})
    h = torch.empty_like(x)
    with pytest.raises(ValueError):
        block_norm_fwd(**ok, residual=h, hidden=h)
    for kw in (dict(x=x, w_pre=w, residual_scale=0.5), dict(x=x), dict(x=x, w_pre=w, residual=h),
               dict(x=x, y=h, hidden=x.clone())):
        with pytest.raises(ValueError):
            block_norm_fwd(**kw)
    g = dict(d_residual=x, d_hidden=x)
    for kw in (dict(g, d_hidden=None), dict(g, d_hidden=x[:5]), dict(g, d_residual=x.float()),
               dict(g, w_pre=None), dict(g, x=x[:5], y=x[:5], d_residual=x[:5], d_hidden=x[:5]),
               dict(g, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            block_norm_bwd(f, **{**ok, **kw})
    with pytest.raises(ValueError):
        block_norm_bwd(BlockNormResult(x, x, torch.empty(2, 5, device="cuda"), 1.0, 1.0, 0.0), **ok, **g)


def test_subnormal_eps_is_refused():
    """The kernel would take it for zero."""
    assert _fwd(eps=1e-42) == 2

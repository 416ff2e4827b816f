"""Refusals of the orthogonalised update, by the wrapper and by the C ABI, before any launch."""

import ctypes

import pytest
import torch

from lm_head_loss_streaming_b200 import _lib, orthogonalize, orthogonalize_workspace_bytes
from orth_util import STANDARD, iterate, spectrum

A = 1 << 20
NAN, INF = float("nan"), float("inf")


def _call(co=None, **kw):
    a = dict(dtype=_lib.SLM_BF16, grad=A, ld=64, stride=64 * 32, batch=2, m=32, n=64,
             momentum=2 * A, beta=0.9, nesterov=True, coefficients=co or [STANDARD] * 5, eps=1e-7,
             out=3 * A, workspace=4 * A, ws_bytes=1 << 30, stream=None)
    a.update(kw)
    return _lib.slm_orthogonalize(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), 4), (dict(m=-1), 2), (dict(n=1 << 30), 2), (dict(batch=65536), 2),
    (dict(m=1 << 29, n=1 << 29, ld=1 << 29), 2), (dict(ld=63), 2), (dict(stride=64 * 32 - 1), 2),
    (dict(eps=0.0), 2), (dict(eps=NAN), 2), (dict(eps=INF), 2), (dict(beta=-0.1), 2),
    (dict(beta=1.1), 2), (dict(beta=NAN), 2), (dict(co=[STANDARD] * 65), 2), (dict(grad=None), 1),
    (dict(out=None), 1), (dict(workspace=None), 1), (dict(grad=A + 1), 3),
    (dict(momentum=2 * A + 2), 3), (dict(out=3 * A + 1), 3), (dict(ws_bytes=1000), 5),
    (dict(workspace=4 * A + 16), 5),
    (dict(co=[(NAN, 0, 0)]), 4), (dict(co=[(1, INF, 0)]), 4), (dict(co=[(2.0, 0, 0)]), 4),
    (dict(co=[(1.8, 0, 0), (1.8, 0, 0)]), 4), (dict(co=[(1.0, 20.0, -20.0)]), 4)])
def test_refusals(kw, status):
    assert _call(**kw) == status


def test_null_coefficients_and_no_steps():
    null = ctypes.POINTER(ctypes.c_float)()
    args = [0, A, 64, 0, 1, 32, 64, None, 0.9, 1, null, 5, 1e-7, A, A, 1 << 30, None]
    assert _lib.load().slm_orthogonalize(*args) == 1
    args[11] = 0
    assert _lib.load().slm_orthogonalize(*args) == 2


def test_empty_stacks_are_fine():
    for kw in (dict(batch=0), dict(m=0), dict(n=0)):
        assert _call(grad=None, out=None, workspace=None, **kw) == _lib.SLM_OK


def test_workspace_bytes():
    assert orthogonalize_workspace_bytes(1, 1 << 30, 4) == 0
    assert orthogonalize_workspace_bytes(-1, 4, 4) == 0
    m, n = 1000, 500
    ws = orthogonalize_workspace_bytes(3, m, n)
    # Three fp16 copies of X (two of hi, one of lo), two of A; some for sums and diagonals.
    assert 3 * 2 * (3 * m * n + 2 * n * n) <= ws <= 3 * 2 * (3 * m * 504 + 2 * n * 504) + (1 << 16)


def test_cpu_tensors_are_refused():
    for g in (torch.zeros(4, 4), torch.zeros(4), None):
        with pytest.raises(ValueError):
            orthogonalize(g)


def test_the_formats_stay_within_what_is_documented():
    """The emulation that the GPU tests take their tolerances from: below 1.5e-3 where a result
    may be off by 2e-3 with its rounding (1.7e-3) included in squares... and 64 bits agree with
    the singular values moved one by one."""
    for kind in ("noise", "decay", "bad", "spikes", "rank"):
        for m, n in ((128, 128), (96, 400), (300, 64)):
            g = spectrum(m, n, kind, 3, "cpu")
            exact = iterate(g, [STANDARD] * 5, 1e-7)
            U, S, Vh = torch.linalg.svd(g / (g.norm() + 1e-7), full_matrices=False)
            for a, b, c in [STANDARD] * 5:
                S = a * S + b * S ** 3 + c * S ** 5
            assert (exact - (U * S) @ Vh).norm() <= 1e-9 * exact.norm()
            off = (iterate(g, [STANDARD] * 5, 1e-7, formats=True) - exact).norm() / exact.norm()
            assert off <= 1.5e-3, (kind, m, n, off)


@pytest.mark.gpu
def test_wrapper_refusals():
    g = torch.zeros(2, 20, 30, device="cuda")
    bad = [dict(grad=g[0, 0]), dict(grad=g.double()), dict(grad=g.transpose(1, 2)),
           dict(grad=g[:1].expand(2, 20, 30)), dict(momentum=g[:, :, :29]),
           dict(momentum=g.bfloat16()), dict(momentum=g), dict(momentum=g.cpu()),
           dict(out=torch.empty_like(g)), dict(out=torch.empty(2, 20, 29, device="cuda").bfloat16()),
           dict(steps=0), dict(steps=65), dict(steps=2, coefficients=[STANDARD] * 3),
           dict(coefficients=(1.0, 2.0)), dict(beta=2.0), dict(eps=0.0),
           dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for kw in bad:
        with pytest.raises(ValueError):
            orthogonalize(**{"grad": g, **kw})
    bf = g.bfloat16()
    with pytest.raises(ValueError):
        orthogonalize(bf, out=bf)
    with pytest.raises(_lib.SLMError):
        orthogonalize(g, coefficients=(3.0, 0.0, 0.0))


def test_subnormal_eps_is_refused():
    """The kernels would take it for zero."""
    assert _call(eps=1e-42) == 2

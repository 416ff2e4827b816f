"""The figures that slm.h gives for how far ``orthogonalize`` may be off the exact iteration, on the
kernels' results: the standard coefficients, five, ten and sixteen steps.

The figures come from rounding in the places where the formats round (``orth_util.iterate`` with
formats, bf16 rounding included) over 4000 matrices of 1 to 600 a side and five kinds of spectra; the
largest found, with both sides 32 or more: 2.2e-3 after five steps, 3.4e-3 after ten and 1.9e-2 after
sixteen at full rank; smaller sides 3.1e-3 after five; low rank or smaller sides 2.1e-2 after ten."""

import pytest
import torch

from lm_head_loss_streaming_b200 import orthogonalize
from orth_util import STANDARD, iterate, spectrum

pytestmark = pytest.mark.gpu
FULL = ("noise", "decay", "bad", "spikes")


def off(g, steps):
    exact = iterate(g, [STANDARD] * steps, 1e-7)
    got = orthogonalize(g, steps=steps).double()
    return (torch.linalg.vector_norm(got - exact) / torch.linalg.vector_norm(exact)).item()


# Matrices in one launch with a side of at most 128, and larger ones; tiles that stay in tensor memory;
# a long axis in parts; wide tiles.
@pytest.mark.parametrize("shape", [(32, 64), (128, 128), (256, 256), (200, 333), (300, 900),
                                   (1000, 700), (40, 5000), (2050, 2100)])
@pytest.mark.parametrize("kind", FULL)
def test_full_rank(shape, kind):
    g = spectrum(*shape, kind, sum(shape)).float()
    for steps, most in ((5, 2.5e-3), (10, 5e-3), (16, 3e-2)):
        e = off(g, steps)
        assert e <= most, (steps, e)


@pytest.mark.parametrize("shape", [(32, 64), (96, 400), (300, 200), (700, 900)])
def test_low_rank(shape):
    g = spectrum(*shape, "rank", sum(shape)).float()
    for steps, most in ((5, 2.5e-3), (10, 3e-2)):
        e = off(g, steps)
        assert e <= most, (steps, e)
    # After more steps the missing directions are there: bounded, whatever they are.
    s = torch.linalg.svdvals(orthogonalize(g, steps=16).double())
    assert s.max() <= 1.3


@pytest.mark.parametrize("shape", [(2, 16), (2, 300), (4, 400), (7, 8), (16, 23), (31, 600), (600, 5)])
@pytest.mark.parametrize("kind", FULL + ("rank",))
def test_narrow(shape, kind):
    for seed in range(5):
        g = spectrum(*shape, kind, seed).float()
        for steps, most in ((5, 4e-3), (10, 3e-2)):
            e = off(g, steps)
            assert e <= most, (seed, steps, e)

"""Which coefficients the orthogonalised update takes: the extremes of the iterates, against the
polynomials sampled closely, and schedules of a polynomial per step on the kernels."""

import random

import numpy as np
import pytest

from lm_head_loss_streaming_b200 import _lib
from orth_util import STANDARD
from test_orth_checks import _call

# A schedule with a polynomial per step: a steep first one, whose iterates reach 1.99, the standard one
# stretched over what that leaves, and the standard one.
SCHEDULE = [(8.287, -23.596, 17.300), tuple(v / 1.75 ** p for v, p in zip(STANDARD, (1, 3, 5))),
            STANDARD, STANDARD]


def extremes(rows):
    """Largest iterate and largest |b s^2 + c s^4| of each step, by samples."""
    most, out = 1.0, []
    for a, b, c in np.float32(rows).astype(np.float64):
        s = np.linspace(0.0, most, 200001)
        pb = b * s ** 2 + c * s ** 4
        most = np.abs(s * (a + pb)).max()
        out.append((most, np.abs(pb).max()))
    return out


def taken(rows):
    """Taken coefficients are refused for the missing gradient behind them (1), others as kind (4)."""
    st = _call(co=[tuple(r) for r in rows], grad=None)
    assert st in (1, 4)
    return st == 1


def test_schedule_with_iterates_near_two_is_taken():
    ext = extremes(SCHEDULE)
    assert 1.99 < max(m for m, _ in ext) < 1.995
    assert taken(SCHEDULE)


def test_limits():
    for top, ok in ((1.99, True), (1.994, True), (1.996, False), (2.0, False), (-1.99, True), (-2.0, False)):
        assert taken([(top, 0.0, 0.0)]) == ok                  # s -> top s, largest at 1
    assert taken([(0.0, 0.0, 0.0)] * 64) and taken([(1.0, 0.0, 0.0)] * 64)
    assert taken([(3.4445, -4.7750, 2.0315)] * 64)


def test_extremes_agree_with_samples():
    rng = random.Random(7)
    seen = [0, 0]
    for _ in range(400):
        rows = []
        for _ in range(rng.randint(1, 4)):
            # A polynomial through (1, p(1)) with a slope of its own; now and then without s^5 or s^3.
            a, b = rng.uniform(-4, 8), rng.uniform(-20, 10)
            c = rng.uniform(-0.5, 2.0) - a - b
            rows.append((a, b if rng.random() < 0.9 else 0.0, c if rng.random() < 0.9 else 0.0))
        ok, near = True, False
        for most, pb in extremes(rows):
            near = near or abs(most - 1.995) < 1e-3 or abs(pb - 15.0) < 1e-2
            if not (most <= 1.995 and pb <= 15.0):
                ok = False
                break
        if not near:
            assert taken(rows) == ok, rows
            seen[ok] += 1
    assert min(seen) >= 20


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 40), (64, 96), (140, 170), (300, 500), (500, 300), (600, 600)])
@pytest.mark.parametrize("kind", ["noise", "decay"])
def test_schedule_on_the_kernels(shape, kind):
    from lm_head_loss_streaming_b200 import orthogonalize
    from orth_util import spectrum
    from test_gpu_orth import check
    g = spectrum(*shape, kind, 3).float()
    for n in range(1, len(SCHEDULE) + 1):
        check(orthogonalize(g, steps=n, coefficients=SCHEDULE[:n]), g, SCHEDULE[:n])
    top = [(1.99, 0.0, 0.0)]
    check(orthogonalize(g, steps=1, coefficients=top), g, top)

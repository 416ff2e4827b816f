"""The number of steps and the coefficients that ``orthogonalize`` makes of its arguments."""

import numpy as np
import pytest

from lm_head_loss_streaming_b200.orth import _steps

ONE = (1.5, -0.5, 0.0)


@pytest.mark.parametrize("steps", [2.5, "5", None, 0, -1, 65, (1,)])
def test_steps_that_are_not_a_whole_number_are_refused(steps):
    for co in (ONE, [ONE] * 5, [ONE] * 2):
        with pytest.raises(ValueError, match="steps"):
            _steps(co, steps)


def test_one_triple_or_one_per_step():
    for steps in (3, 3.0, np.int64(3)):
        assert _steps(ONE, steps) == [ONE] * 3 == _steps([ONE] * 3, steps)
    for bad in ([ONE] * 2, [ONE] * 4, (1.0, 2.0), [(1.0, 2.0)] * 3, []):
        with pytest.raises(ValueError, match="coefficients"):
            _steps(bad, 3)

"""The float64 definition of the recurrence where gates are nearly open or closed."""

import numpy as np
import pytest

from oracle import recurrent_oracle as ro


@pytest.mark.parametrize("i", [-60.0, -30.0, 0.0, 5.0, 30.0, 60.0])
def test_gradient_of_an_open_input_gate(i):
    """One token without a state: h = x sigma(i), dL/di = x sigma(i) sigma(-i), which has all of its digits."""
    x = np.full((1, 1), 3.0)
    got = ro.gated_backward64(x, np.zeros((1, 1)), np.ones((1, 1)), None, np.full((1, 1), i), scale="none")
    # sigma(i) sigma(-i) = 1 / (2 + 2 cosh i)
    assert abs(got["dinput_gate"][0, 0] * (2.0 + 2.0 * np.cosh(i)) - 3.0) <= 1e-14

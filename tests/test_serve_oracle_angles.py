"""The fp64 statement of the rotation against whole turns taken out in exact fractions, for every frequency that
the call takes. An angle below pi in 64 bits is off by four roundings at most (2^-53 of pi each): 2e-15."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import serve

TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256")


@pytest.mark.parametrize("pos", [0, 1, -5, 131071, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("freq", [1.0, 0.123456, -0.3, 1e-6, 1e-45, 100000.25, 2.0 ** 23 + 1, 2.0 ** 24 - 1])
def test_far_and_fast_angles(pos, freq):
    f = np.float32(freq)
    t = Fraction(float(f)) * pos
    t = float(t - TWO_PI * round(t / TWO_PI))
    u = np.zeros((1, 1, 2))
    u[0, 0, 0] = 1.0
    got, size = serve.turn(u, [pos], [f], False)
    np.testing.assert_allclose(got[0, 0], [np.cos(t), np.sin(t)], rtol=0, atol=2e-15)
    assert (size == 1).all()

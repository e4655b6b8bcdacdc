"""The rotation's angle, seen through heads that it turns onto an axis.

The pair (a, b) = (sin t, cos t) turned by t is (a cos t - b sin t, b cos t + a sin t) = (0, 1), so the first
element is what is missing of the angle, and its rounding to bf16 relative to that. Bound for it:
  pi 2^-25          the angle in half turns rounded to fp32 (below 1: 2^-25)
  sqrt2 2^-25       a and b given in fp32
  2 sqrt2 2^-25     sine and cosine off by a step (2^-24 below 1)
  2^-25             the rounding of b sin t
  2 pi 2^-31        whole turns dropped from a 64-bit fraction, its upper 32 bits taken
times 1 + 2^-8.
"""
from fractions import Fraction

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256")
BOUND = ((np.pi + 3 * 2 ** 0.5 + 1) * 2.0 ** -25 + 2 * np.pi * 2.0 ** -31) * (1 + 2.0 ** -8)


def angles(pos, f):
    """pos * f without its whole turns, between -pi and pi, in 64 bits."""
    t = np.empty((len(pos), len(f)))
    for i, p in enumerate(pos):
        for j, x in enumerate(f):
            r = Fraction(float(x)) * int(p)
            t[i, j] = float(r - TWO_PI * round(r / TWO_PI))
    return t


POS = [0, 1, -1, 2, 4095, 131071, 131072, 2 ** 24 + 1, 123456789, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345]
FREQS = {
    "usual": 1e6 ** (-np.arange(32) / 32),
    "up to one": 1 - np.arange(32) * 0.03,
    "large": [7.0, 100.5, 1000.1, 100000.25, 2.0 ** 20 + 0.125, 2.0 ** 23 - 0.5, 2.0 ** 23 + 1, 2.0 ** 24 - 1] * 4,
    "small and negative": [0.0, -0.3, -1.0, 2e-12, 1e-30, 1e-45, -2.0 ** 23 - 1, -99.9] * 4,
}


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("which", list(FREQS))
def test_angle(which, pairs):
    import torch
    import bit_weight_only_w4a16_gb300 as w4
    w4.init()
    f = np.asarray(FREQS[which], np.float32)
    t = angles(POS, f)
    a, b = np.float32(np.sin(t)), np.float32(np.cos(t))
    i = np.arange(32) * (2 if pairs else 1)
    j = i + (1 if pairs else 32)
    q = np.zeros((len(POS), 1, 64), np.float32)
    q[:, 0, i], q[:, 0, j] = a, b
    pos = torch.tensor(POS, dtype=torch.int32, device="cuda")
    out, _ = w4.w4_qk_norm_rope(torch.from_numpy(q).cuda(), None, pos, torch.from_numpy(f).cuda(), pairs=pairs)
    got = out.double().cpu().numpy()[:, 0]
    worst = np.abs(got[:, i]).max(0)
    assert (worst <= BOUND).all(), f"{dict(zip(f.tolist(), (worst / BOUND).round(2).tolist()))}"
    assert (np.abs(got[:, j] - 1) <= 2.0 ** -8).all()

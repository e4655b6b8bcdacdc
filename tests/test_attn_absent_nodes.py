"""Absent nodes beside NaN and infinities in values that the present nodes keep: an
absent node's row is zeros whatever the others see."""
import numpy as np
import pytest

import synth
from test_attn_tree_parity import make, run, w4  # noqa: F401

pytestmark = pytest.mark.gpu


# B = 1: the one row tile is cut over several CTAs; B = 320: more row tiles than SMs, whole ones.
@pytest.mark.parametrize("B,T", [(1, 700), (320, 24)])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("ring", [False, True])
def test_absent_rows_are_zero(w4, B, T, D, ring):  # noqa: F811
    N, Hq, Hkv = 5, 4, 2
    parents = np.tile(np.array([[-1, 0, -2, 1, -2]], np.int32), (B, 1))
    pos = np.full(B, T, np.int32)
    kpos = np.stack([synth.ring_positions(T - 1, T)] * B) if ring else None
    t = make(50 + D, B, N, T, Hq, Hkv, D)
    clean = run(w4, *t, parents, pos, kpos, 0, D ** -0.5)
    assert not clean[:, [2, 4]].any() and np.isfinite(clean).all()
    t[2][:, 5, 0, 3] = float("nan")   # head 0: query heads 0 and 1
    t[2][:, T - 1, 1, 10] = float("inf")
    t[4][:, 0, 1, 20] = float("-inf")  # the first node, which every present node keeps
    got = run(w4, *t, parents, pos, kpos, 0, D ** -0.5)
    assert not got[:, [2, 4]].any()
    here = got[:, [0, 1, 3]]
    assert np.isnan(here[:, :, :2, 3]).all()
    assert (here[:, :, 2:, 10] == np.inf).all() and (here[:, :, 2:, 20] == -np.inf).all()
    want = clean[:, [0, 1, 3]].copy()
    want[:, :, :2, 3], want[:, :, 2:, 10], want[:, :, 2:, 20] = np.nan, np.inf, -np.inf
    np.testing.assert_array_equal(here, want)

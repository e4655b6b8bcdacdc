"""More row tiles than a block has threads (the cutting of the work takes several
rounds) and than the GPU has SMs (row tiles count with their fixed cost)."""
import numpy as np
import pytest

import test_attn_prompt_parity as prompt
import test_attn_tree_parity as tree
from oracle import draft
from test_attn_prompt_parity import w4  # noqa: F401

pytestmark = pytest.mark.gpu


# 128 query heads on one: one token per 128 rows, so one or two tokens a row tile.
@pytest.mark.parametrize("D", [64, 128, 256, 384, 512])
@pytest.mark.parametrize("lq,lk,window", [([900], [900], 40), ([500, 0, 1, 250, 149], [520, 7, 300, 250, 0], 0),
                                          ([811], [1500], 200)])
def test_prompt(w4, D, lq, lk, window):  # noqa: F811
    Hq, heads = 128, [0, 77, 127]
    q, k, v, cu_q, cu_k = prompt.make(sum(lq) + D, lq, lk, Hq, 1, D)
    got = prompt.run(w4, q, k, v, cu_q, cu_k, window, D ** -0.5)[:, heads]
    assert np.isfinite(got).all()
    qf, kf, vf = (x.float().numpy().astype(np.float64) for x in (q[:, heads], k, v))
    ref, ab = draft.attn_prompt(qf, kf, vf, cu_q, cu_k, window, D ** -0.5)
    S = D ** -0.5 * float(np.sqrt((qf ** 2).sum(-1).max() * (kf ** 2).sum(-1).max()))
    err, bound = np.abs(got - ref), prompt.rel_bound(D, S, max(lk)) * ab + 1e-30
    assert (err <= bound).all(), f"worst ratio {(err / bound).max():.3f}"


@pytest.mark.parametrize("D", [64, 256, 512])
def test_tree_batch(w4, D):  # noqa: F811
    rng = np.random.default_rng(D)
    B, T = 450, 20
    pos = rng.integers(0, T + 1, B)
    parents = np.full((B, 1), -1, np.int32)
    parents[::7] = -2
    got = tree.check(w4, D, B, 1, T, 2, 1, D, parents, pos)
    assert not got[::7].any()

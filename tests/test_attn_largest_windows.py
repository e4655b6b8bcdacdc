"""Windows up to 2^31 - 1 cut nothing: the same bits as without a window."""
import numpy as np
import pytest

import synth
import test_attn_prompt_parity as prompt
import test_attn_tree_parity as tree
from test_attn_prompt_parity import w4  # noqa: F401

pytestmark = pytest.mark.gpu

WINDOWS = [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 31 - 257]


@pytest.mark.parametrize("window", WINDOWS)
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_prompt(w4, D, window):  # noqa: F811
    """Also with more queries than keys, where positions begin below zero."""
    q, k, v, cu_q, cu_k = prompt.make(D, [200, 30, 257], [100, 190, 1], 8, 2, D)
    want = prompt.run(w4, q, k, v, cu_q, cu_k, 0, D ** -0.5)
    assert want[100:200].any(-1).all() and not want[:100].any() and want[230 + 256].any()
    np.testing.assert_array_equal(prompt.run(w4, q, k, v, cu_q, cu_k, window, D ** -0.5), want)


@pytest.mark.parametrize("window", WINDOWS)
@pytest.mark.parametrize("ring", [False, True])
def test_tree(w4, ring, window):  # noqa: F811
    T, N, D, pos = 300, 12, 128, 290
    t = tree.make(3, 1, N, T, 8, 2, D)
    parents = np.arange(-1, N - 1, dtype=np.int32)[None]
    kpos = synth.ring_positions(pos - 1, T)[None] if ring else None
    want = tree.run(w4, *t, parents, [pos], kpos, 0, D ** -0.5)
    np.testing.assert_array_equal(tree.run(w4, *t, parents, [pos], kpos, window, D ** -0.5), want)

"""Sequence bounds that are not ascending: nothing outside the tensors is read or
written, an end before its start is an empty sequence."""
import numpy as np
import pytest

import test_attn_prompt_parity as prompt
from _guard import Guard
from test_attn_prompt_parity import w4  # noqa: F401

pytestmark = pytest.mark.gpu

LEAST = -2 ** 31


@pytest.mark.parametrize("cu", [[1, LEAST], [5, 3], [2 ** 31 - 1, LEAST], [-1, 5], [0, LEAST, LEAST, 0]])
@pytest.mark.parametrize("D", [128, 256])
def test_queries(w4, D, cu):  # noqa: F811
    import torch
    q, k, v, _, _ = prompt.make(1, [6], [6], 4, 1, D)
    g = Guard((6, 4, D), torch.bfloat16)
    g.t.fill_(5.0)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ck = torch.arange(0, len(cu), dtype=torch.int32, device="cuda")
    w4.w4_attn_prompt(q.cuda(), k.cuda(), v.cuda(), c, ck, out=g.t)
    torch.cuda.synchronize()
    g.check("w4_attn_prompt")
    assert bool((g.t == 5.0).all()) and w4.device_error() == 0


@pytest.mark.parametrize("cu", [[1, LEAST], [5, 3], [2 ** 31 - 1, LEAST], [2 ** 31 - 1, 2 ** 31 - 1], [3, 3]])
@pytest.mark.parametrize("D", [128, 256])
def test_keys(w4, D, cu):  # noqa: F811
    q, k, v, _, _ = prompt.make(2, [6], [6], 4, 1, D)
    got = prompt.run(w4, q, k, v, np.array([0, 6], np.int32), np.array(cu, np.int32), 0, 0.1)
    assert not got.any()

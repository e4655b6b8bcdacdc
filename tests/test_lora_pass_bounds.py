"""Adapters of more rows than the scratch holds partial sums of: rows around the end of a pass, and last passes
short enough to be ranked like a decode batch (their rows begin past zero).

The scratch has 2 SMs (32768 + 512) + 8 SMs + 64 floats, and 8 MB at least; a pass takes the rows whose R floats fit it,
in whole tiles of 64. Bound, elementwise, with low = |s| sum_r |b| sum_k |a x|: 2^-24 |out| (one addition to y) and
(K + 3 R + 82) 2^-23 low (sums of K and 3 R products, each addition off by a step at most).
"""
import numpy as np
import pytest

from _guard import Guard

pytestmark = pytest.mark.gpu

R, K, N, L = 128, 32, 8, 3


@pytest.fixture(scope="module")
def w4():
    import bit_weight_only_w4a16_gb300 as w4
    w4.init()
    return w4


def rows_of_a_pass():
    import torch
    n = torch.cuda.get_device_properties(0).multi_processor_count
    return max(2 * n * 32768 + 2 * n * 512 + 8 * n + 64, 1 << 21) // R // 64 * 64


@pytest.mark.parametrize("behind", [1, 300, 512, 513, 1200])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_around_the_end_of_a_pass(w4, behind, in_place):
    import torch
    first = rows_of_a_pass()
    M = first + behind
    g = torch.Generator(device="cuda").manual_seed(behind)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")
    y, x = randn(M, N), randn(M, K).bfloat16()
    a, b, s = (randn(L, R, K) * K ** -0.5).bfloat16(), (randn(L, N, R) * 0.3).bfloat16(), 0.5 + torch.rand(L, generator=g,
                                                                                                        device="cuda")
    ids = np.repeat([0, -1, 2], [first - 100, 40, M - first + 60])  # the last adapter's rows lie in both passes
    ids[-behind // 2 - 1:] = 1
    out = Guard((M, N), torch.float32)
    out.t.copy_(y)
    w4.w4_lora(out.t if in_place else y, x, a, b, torch.from_numpy(ids.astype(np.int32)).cuda(), scale=s, out=out.t)
    torch.cuda.synchronize()
    out.check("out")
    got, yy, xx, aa, bb, ss = (t.double().cpu().numpy() for t in (out.t, y, x, a, b, s))
    live = ids >= 0
    ref, low = yy.copy(), np.zeros_like(yy)
    for i in range(L):
        m = ids == i
        ref[m] += ss[i] * (xx[m] @ aa[i].T @ bb[i].T)
        low[m] = ss[i] * (np.abs(xx[m]) @ np.abs(aa[i]).T @ np.abs(bb[i]).T)
    bound = 2.0 ** -24 * np.abs(ref) + (K + 3 * R + 82) * 2.0 ** -23 * low
    assert (np.abs(got - ref) <= bound)[live].all()
    np.testing.assert_array_equal(got[~live], yy[~live])

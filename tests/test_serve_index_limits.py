"""The serving calls on tensors of more than 2^31 elements: the last rows and adapters against the same ones in
small tensors of their own."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import bit_weight_only_w4a16_gb300 as w4
    w4.init()
    return w4


def randn(seed, *s):
    import torch
    return torch.randn(*s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def test_projections_past_32_bits(w4):
    """Adapters on 2.2e9 elements of y, in place: the last rows, those around element 2^31, and one without an adapter."""
    import torch
    M, N, K, R = 270000, 8192, 32, 8
    a, b = (randn(1, 2, R, K) * K ** -0.5).bfloat16(), randn(2, 2, N, R).bfloat16()
    x = randn(3, M, K).bfloat16()
    y = torch.zeros(M, N, device="cuda")
    assert y.numel() > 1 << 31
    ids = np.repeat([0, 1, -1, 1], [200000, 65000, 10, M - 265010])
    w4.w4_lora(y, x, a, b, i32(ids), out=y)
    for m in (slice(0, 40), slice(262130, 262160), slice(264990, 265020), slice(M - 700, M)):
        n = m.stop - m.start
        want = w4.w4_lora(torch.zeros(n, N, device="cuda"), x[m].contiguous(), a, b, i32(ids[m]))
        torch.testing.assert_close(y[m], want, rtol=0, atol=2.0 ** -18 * float(want.abs().max()))
        assert (y[m].abs().sum(1) > 0).tolist() == (ids[m] >= 0).tolist()


@pytest.mark.parametrize("M", [5, 600])
def test_adapters_past_32_bits(w4, M):
    import torch
    L, R, N, K = 1100, 128, 16384, 16384
    a, b = (torch.zeros(L, *s, dtype=torch.bfloat16, device="cuda") for s in ((R, K), (N, R)))
    assert a.numel() > 1 << 31 and b.numel() > 1 << 31
    at = [0, 1023, 1024, L - 1]
    for i in at:
        a[i], b[i] = (randn(i, R, K) * K ** -0.5).bfloat16(), randn(i + 1, N, R).bfloat16()
    x, y = randn(5, M, K).bfloat16(), randn(6, M, N)
    pick = np.repeat(np.arange(4), -(-M // 4))[:M]
    got = w4.w4_lora(y, x, a, b, i32(np.array(at)[pick]))
    want = w4.w4_lora(y, x, a[at].contiguous(), b[at].contiguous(), i32(pick))
    assert torch.equal(got, want)
    assert float((got - y).abs().max()) > 1


def test_heads_past_32_bits(w4):
    import torch
    M, Hq, Hkv, D = 34000, 126, 2, 512
    q = torch.zeros(M, Hq, D, dtype=torch.bfloat16, device="cuda")
    assert q.numel() > 1 << 31
    k = randn(1, M, Hkv, D).bfloat16()
    rows = [0, 33287, 33288, M - 1]
    for m in rows:
        q[m] = randn(m, Hq, D).bfloat16()
    pos, f, w = i32(np.arange(M) + 70000), torch.linspace(1, 0.001, D // 2, device="cuda"), 1 + 0.2 * randn(2, D)
    out, ko = w4.w4_qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w)
    want, kw = w4.w4_qk_norm_rope(q[rows].contiguous(), k[rows].contiguous(), pos[rows].contiguous(), f, q_weight=w, k_weight=w)
    assert torch.equal(out[rows], want) and torch.equal(ko[rows], kw)
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert all(not bool(part.any()) for part in out[rest].split(4000))
    # in place
    w4.w4_qk_norm_rope(q, None, pos, f, q_weight=w, q_out=q)
    assert torch.equal(q[rows], want)

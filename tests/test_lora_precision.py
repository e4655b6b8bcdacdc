"""The adapters' stated precision, with values whose sums are exact or whose bound is tight.

h = a x goes to the second product as three bf16 parts. Every rounding to bf16 is off by at most 2^-8 of the
value, so three leave 2^-24 of h, two would leave 2^-16.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import bit_weight_only_w4a16_gb300 as w4
    w4.init()
    return w4


def dev(a, dt=np.float32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()


def bf16(x):
    """x rounded to bf16 (to nearest, ties to even), in 64 bits."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def exact_rows(rng, M, K, R, L):
    """x [M][K], a [L][R][K] (values that bf16 holds) and h [M][L][R], exact in 24 bits: a x is the sum of three products,
    an integer below 2^24 with its upper 8 bits in 128 .. 253, times 2^-16."""
    x, a = np.zeros((M, K)), np.zeros((L, R, K))
    at = rng.permutation(K)[:3]
    p = np.stack([rng.integers(128, 254, (L, R)), rng.integers(0, 256, (L, R)), rng.integers(0, 256, (L, R))], -1)
    a[:, :, at] = p
    sign = rng.choice([-1.0, 1.0], M)
    x[:, at] = sign[:, None] * np.array([1.0, 2.0 ** -8, 2.0 ** -16])
    return x, a, sign[:, None, None] * (p @ np.array([1.0, 2.0 ** -8, 2.0 ** -16]))[None]


@pytest.mark.parametrize("M", [1, 40, 300, 700])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 72, 128])
def test_three_parts(w4, M, R):
    """Every column takes one element of h, times a power of two, onto y = 0: all sums are exact (each has one
    product, or three whose bits end at 2^-16 and lie below 2^8), so the parts' 2^-24 is all that may be missing."""
    rng = np.random.default_rng(R + M)
    K, L, N = 64, 3, 128
    x, a, h = exact_rows(rng, M, K, R, L)
    pick = rng.integers(0, R, (L, N))
    b = np.zeros((L, N, R))
    b[np.arange(L)[:, None], np.arange(N)[None], pick] = 2.0 ** rng.integers(-3, 4, (L, N))
    ids = np.repeat(np.arange(L), -(-M // L))[:M] if M > 512 else rng.integers(0, L, M)
    scale = 2.0 ** rng.integers(-2, 3, L)
    ref = np.einsum("mnr,mr->mn", b[ids], h[np.arange(M), ids]) * scale[ids][:, None]
    got = w4.w4_lora(dev(np.zeros((M, N))), dev(x).bfloat16(), dev(a).bfloat16(), dev(b).bfloat16(), dev(ids, np.int32),
                     scale=dev(scale)).double().cpu().numpy()
    bound = 2.0 ** -24 * np.abs(ref)
    assert (np.abs(got - ref) <= bound).all(), f"worst {(np.abs(got - ref) / np.abs(ref)).max():.3g}"
    # What two parts would leave is seen here.
    two = bf16(ref) + bf16(ref - bf16(ref))
    assert (np.abs(two - ref) > 16 * bound).any()


@pytest.mark.parametrize("M", [1, 40, 300, 700])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 72, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_added_to_y_once(w4, M, R, in_place):
    """Large projections with small adapters: one rounding of the sum, 2^-24 |out| (its half step), and the adapters' own sum,
    formed apart: with low = |s| sum_r |b| sum_k |a x|
      2^-24 low                h's parts
      (K + 3 R + 80) 2^-23 low  sums of K and of 3 R products, of warps and blocks, and the scale, each addition off by a step
    Products added to y one after another would each be rounded at y's magnitude."""
    rng = np.random.default_rng(R + M)
    K, L, N = 32, 3, 128
    y = np.float32(rng.choice([-1.0, 1.0], (M, N)) * 2.0 ** (16 + rng.random((M, N))))
    x, a = bf16(rng.standard_normal((M, K))), bf16(rng.standard_normal((L, R, K)) * K ** -0.5)
    b = bf16(rng.standard_normal((L, N, R)) * 0.1)
    ids = np.repeat(np.arange(L), -(-M // L))[:M] if M > 512 else rng.integers(0, L, M)
    scale = np.float32(0.5 + rng.random(L))
    h = np.einsum("lrk,mk->mlr", a, x)[np.arange(M), ids]
    ha = np.einsum("lrk,mk->mlr", np.abs(a), np.abs(x))[np.arange(M), ids]
    s = scale.astype(np.float64)[ids][:, None]
    ref = y.astype(np.float64) + s * np.einsum("mnr,mr->mn", b[ids], h)
    low = s * np.einsum("mnr,mr->mn", np.abs(b)[ids], ha)
    ty = dev(y)
    got = w4.w4_lora(ty, dev(x).bfloat16(), dev(a).bfloat16(), dev(b).bfloat16(), dev(ids, np.int32), scale=dev(scale),
                     out=ty if in_place else None).double().cpu().numpy()
    bound = 2.0 ** -24 * np.abs(ref) + (K + 3 * R + 82) * 2.0 ** -23 * low
    err = np.abs(got - ref)
    assert (err <= bound).all(), f"worst {(err / bound).max():.3f}"


@pytest.mark.parametrize("M", [40, 700])
def test_rows_without_an_adapter_keep_their_bits(w4, M):
    import torch
    y = torch.randn(M, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(M))
    y[:, ::3] = -0.0
    y[:, 1::9] = float("nan")
    x, a, b = (torch.ones(s, dtype=torch.bfloat16, device="cuda") for s in ((M, 32), (2, 8, 32), (2, 64, 8)))
    ids = np.arange(M) % 3 - 1
    out = w4.w4_lora(y, x, a, b, dev(ids, np.int32))
    none = torch.from_numpy(ids < 0).cuda()
    assert torch.equal(out[none].view(torch.int32), y[none].view(torch.int32))

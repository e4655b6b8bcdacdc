"""Single tokens over a paged cache at the precision that the call states: weights in two bf16 parts.

Elementwise bound, times sum_t w_t |v_t| where nothing else is said:
  2^-8 |out|       the output rounded to bf16 (half a step)
  2^-16            a weight in two parts, each off by 2^-8 of what it rounds
  2^-15            exp2 of the hardware and the rounding of its argument
  8 2^-23 S        queries and keys are whole numbers, so scores are exact: the scale's two roundings and the
                   score's, the subtraction of the maximum, of both scores (S = max of scale * |q| |k|)
  (T/8 + 64) 2^-23 the fp32 accumulation over T keys, the rescales and the joins
A weight in one part is off by up to 2^-8: where the values nearly cancel, that is seen.
"""
import numpy as np
import pytest

from oracle import serve
from test_attn_paged_parity import Batch, dev, f64, w4  # noqa: F401

pytestmark = pytest.mark.gpu


def bf16(x):
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def one_part(q, k, v, table, lens, page, scale):
    """The attention with each weight, relative to the largest, rounded to bf16 once: what must not pass."""
    M, Hq, D = q.shape
    G = Hq // k.shape[2]
    out = np.zeros((M, Hq, D))
    for b in range(M):
        n = int(lens[b])
        if n == 0:
            continue
        t = np.arange(n)
        g = table[b, t // page]
        for h in range(Hq):
            s = k[g, t % page, h // G] @ q[b, h] * scale
            w = np.exp(s - s.max())
            out[b, h] = bf16(w) @ v[g, t % page, h // G] / w.sum()
    return out


def tight(w4, b, window=0, sees_one_part=True):  # noqa: F811
    D = b.q.shape[2]
    for t in (b.q, b.k):
        t.copy_(t.float().round().clamp(-3, 3))
    scale = D ** -0.5
    got = b.run(w4, window, scale, step=True)
    q, k, v = f64(b.q), f64(b.k), f64(b.v)
    ref, ab = serve.attn_paged(q, k, v, b.table, b.lens, None, window, scale)
    S = scale * float(np.sqrt((q ** 2).sum(-1).max() * (k ** 2).sum(-1).max()))
    T = max(1, int(b.lens.max()))
    rel = 2.0 ** -16 + 2.0 ** -15 + 8 * 2.0 ** -23 * S + (T / 8 + 64) * 2.0 ** -23
    bound = 2.0 ** -8 * np.abs(ref) + (rel * ab + 1e-30) * (1 + 2.0 ** -8)
    err = np.abs(got - ref)
    assert (err <= bound).all(), f"worst ratio {(err / bound).max():.3f}"
    if sees_one_part:
        one = one_part(q, k, v, b.table, b.lens, b.page, scale)
        assert (np.abs(one - ref) > 2 * bound).any()
    return got


SHAPES = [(64, 8, 1), (64, 16, 1), (128, 8, 2), (128, 11, 1), (256, 8, 1), (256, 16, 1), (384, 6, 2), (512, 8, 1)]


@pytest.mark.parametrize("D,Hq,Hkv", SHAPES)
def test_two_parts(w4, D, Hq, Hkv):  # noqa: F811
    """Short tables: whole segments, with few of them shared by a cluster's blocks."""
    for B in (1, 3, 170):
        lens = np.random.default_rng(B + D).integers(2, 40, B)
        tight(w4, Batch(B + D, np.ones(B, int), lens, Hq, Hkv, D, 16))


@pytest.mark.parametrize("D,Hq,Hkv", SHAPES)
def test_tables_much_wider_than_the_lengths(w4, D, Hq, Hkv):  # noqa: F811
    """A table with room for 16000 positions: runs are cut as if the segments were long, and joined."""
    for B in (1, 3, 61):
        lens = np.random.default_rng(B + D).integers(0, 40, B)
        lens[0] = 2
        b = Batch(B + D, np.ones(B, int), lens, Hq, Hkv, D, 16, extra_cols=1000)
        got = tight(w4, b)
        assert not got[lens == 0].any()
        narrow = Batch(B + D, np.ones(B, int), lens, Hq, Hkv, D, 16)
        tight(w4, narrow)
    lens = np.array([0, 3000, 1, 700, 16])
    tight(w4, Batch(D, np.ones(5, int), lens, Hq, Hkv, D, 16, extra_cols=900), sees_one_part=False)
    tight(w4, Batch(D, np.ones(5, int), lens, Hq, Hkv, D, 16, extra_cols=900), window=100, sees_one_part=False)


@pytest.mark.parametrize("wide", [0, 64])
def test_single_tokens_of_a_pool_past_32_bits(w4, wide):  # noqa: F811
    """Pages whose elements lie past 2^31 in the pool, on tables as wide as the lengths and wider."""
    import torch
    pages, page = 16500, 1024
    k = torch.zeros(pages, page, 1, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    for window in (0, 300):
        b = Batch(21, [1, 1], [1500, 1024], 8, 1, 128, page, spare=0, extra_cols=wide)
        far = np.array([pages - 1, 3, pages - 2])
        k[torch.from_numpy(far).cuda()], v[torch.from_numpy(far).cuda()] = b.k, b.v
        want = b.run(w4, window, step=True)
        b.check(w4, window, step=True)
        b.k, b.v = k, v
        b.table = np.where(b.table >= 0, far[np.maximum(b.table, 0)], -1).astype(np.int32)
        np.testing.assert_array_equal(b.run(w4, window, step=True), want)
    t = 1023  # the last key of sequence 1, in a page past 2^31 elements or the third
    v[b.table[1, 0], t, 0, 3] = float("nan")
    got = b.run(w4, window, step=True)
    assert np.isnan(got[1, :, 3]).all() and np.isfinite(np.delete(got, 3, 2)).all() and np.isfinite(got[0]).all()

"""Low-rank adapters against the fp64 statement.

Elementwise bound, derived from the kernel's arithmetic. With low = |s| sum_r |b| |h| and
size = |y| + |s| sum_r |b| sum_k |a x| (low <= size):
  2^-18 low            h carried as two bf16 parts (hi within 2^-8 of h, lo within 2^-8 of the
                       rest: 2^-16; the rounding of lo is 2^-17 of h at most), taken as 2^-16 low
  (K + 2 R + 40) 2^-24 size   fp32 sums of exact products: K additions for h, then its parts', the
                       scale, 2 R additions onto y
"""
import numpy as np
import pytest

from _guard import Guard
from oracle import serve

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import bit_weight_only_w4a16_gb300 as w4
    w4.init()
    return w4


def dev(a, dt=np.int32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()


def make(seed, M, N, K, R, L):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")
    return (randn(M, N), randn(M, K).bfloat16(), (randn(L, R, K) * K ** -0.5).bfloat16(), (randn(L, N, R) * 0.3).bfloat16(),
            0.5 + torch.rand(L, generator=g, device="cuda"))


def check(w4, y, x, a, b, ids, scale, in_place=False):
    import torch
    M, N = y.shape
    L, R, K = a.shape
    g = Guard((M, N), torch.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y0 = y.clone()
    if in_place:
        g.t.copy_(y)
        w4.w4_lora(g.t, x, a, b, dev(ids), scale=scale, out=g.t, status=st)
    else:
        w4.w4_lora(y, x, a, b, dev(ids), scale=scale, out=g.t, status=st)
    torch.cuda.synchronize()
    g.check("w4_lora")
    assert torch.equal(y, y0)
    got = g.t.double().cpu().numpy()
    ref, size, low, status = serve.lora(y.cpu().numpy(), x.float().cpu().numpy(), a.float().cpu().numpy(),
                                        b.float().cpu().numpy(), ids, None if scale is None else scale.cpu().numpy())
    bound = 2.0 ** -16 * low + (K + 2 * R + 40) * 2.0 ** -24 * size
    err = np.abs(got - ref)
    assert np.isfinite(got).all() and (err <= bound).all(), f"worst {(err / np.maximum(bound, 1e-300)).max():.3f}"
    assert int(st) == status
    none = np.array([not 0 <= i < L for i in ids])
    np.testing.assert_array_equal(got[none], y0.double().cpu().numpy()[none])
    return g.t


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 96, 120, 128])
@pytest.mark.parametrize("M", [1, 5, 100])
def test_ranks(w4, R, M):
    rng = np.random.default_rng(R + M)
    check(w4, *make(R, M, 264, 96, R, 5)[:4], rng.integers(-1, 5, M), make(R, 1, 8, 32, 8, 5)[4])


@pytest.mark.parametrize("R", [8, 32, 72, 128])
def test_ranks_of_prompts(w4, R):
    """More rows than are ranked: tiles of 64 rows in order, adapters in runs and mixed."""
    y, x, a, b, s = make(R + 1, 700, 72, 256, R, 6)
    runs = np.repeat([0, 3, -1, 5, 3], [130, 1, 63, 400, 106])
    check(w4, y, x, a, b, runs, s)
    check(w4, y, x, a, b, np.random.default_rng(R).integers(-1, 6, 700), s)


@pytest.mark.parametrize("M", [16, 17, 64, 255, 256, 257, 511, 512, 513])
def test_rows_around_the_limits(w4, M):
    rng = np.random.default_rng(M)
    y, x, a, b, s = make(M, M, 64, 64, 16, 7)
    for ids in (np.zeros(M, int), np.full(M, -1), rng.integers(-1, 7, M), np.arange(M) % 7, rng.integers(0, 2, M) * 6):
        check(w4, y, x, a, b, ids, s)


@pytest.mark.parametrize("N,K", [(8, 32), (2048, 1536), (248, 6144), (12288, 1536), (256, 32), (1000, 4096)])
def test_shapes(w4, N, K):
    y, x, a, b, s = make(N, 19, N, K, 16, 3)
    check(w4, y, x, a, b, np.arange(19) % 4 - 1, s)


@pytest.mark.parametrize("N,K", [(24, 96), (40, 608), (520, 4128), (2048, 32)])
def test_shapes_of_prompts(w4, N, K):
    """Columns and summed elements that end within a step of the kernels."""
    y, x, a, b, s = make(N + 1, 777, N, K, 24, 3)
    check(w4, y, x, a, b, np.repeat([1, -1, 2, 0], [400, 7, 300, 70]), s)


def test_many_adapters(w4):
    y, x, a, b, s = make(1, 300, 40, 64, 8, 500)
    ids = np.random.default_rng(2).integers(0, 500, 300)
    check(w4, y, x, a, b, ids, s)
    check(w4, y, x, a, b, ids[::-1].copy(), None)


def test_ids_that_are_none(w4):
    y, x, a, b, s = make(3, 20, 64, 64, 8, 2)
    check(w4, y, x, a, b, np.array([0, 2, 1, -2**31, 2**31 - 1] * 4), s)
    check(w4, y, x, a, b, np.full(20, 9), s)
    y, x, a, b, s = make(3, 600, 64, 64, 8, 2)
    check(w4, y, x, a, b, np.array([0, 2, 1, -5, 1] * 120), s)


@pytest.mark.parametrize("M", [7, 600])
def test_in_place_and_strided(w4, M):
    import torch
    rng = np.random.default_rng(M)
    y, x, a, b, s = make(4, M, 96, 128, 32, 4)
    ids = rng.integers(-1, 4, M)
    want = check(w4, y, x, a, b, ids, s)
    assert torch.equal(check(w4, y, x, a, b, ids, s, in_place=True), want)
    wide = torch.full((M, 256), 7.0, device="cuda")
    wide[:, 64:160] = y
    xw = torch.zeros(M, 200, dtype=torch.bfloat16, device="cuda")
    xw[:, 8:136] = x
    w4.w4_lora(wide[:, 64:160], xw[:, 8:136], a, b, dev(ids), scale=s, out=wide[:, 64:160])
    assert torch.equal(wide[:, 64:160], want)
    assert bool((wide[:, :64] == 7).all()) and bool((wide[:, 160:] == 7).all())


def test_rows_do_not_reach_each_other(w4):
    """NaN in one row's x, or in an adapter, stays with its rows."""
    import torch
    for M in (40, 600):
        y, x, a, b, s = make(5, M, 64, 64, 16, 4)
        ids = np.arange(M) % 5 - 1
        want = w4.w4_lora(y, x, a, b, dev(ids), scale=s)
        x2 = x.clone()
        x2[9] = float("nan")
        got = w4.w4_lora(y, x2, a, b, dev(ids), scale=s)
        assert torch.isnan(got[9]).all()
        got[9] = want[9]
        assert torch.equal(got, want)
        a2 = a.clone()
        a2[2] = float("inf")
        got = w4.w4_lora(y, x, a2, b, dev(ids), scale=s)
        rest = torch.from_numpy(ids != 2).cuda()
        assert not torch.isfinite(got[~rest]).any() and torch.equal(got[rest], want[rest])
        b2 = b.clone()
        b2[2, 5:9] = float("nan")
        got = w4.w4_lora(y, x, a, b2, dev(ids), scale=s)
        assert torch.isnan(got[~rest][:, 5:9]).all() and torch.equal(got[rest], want[rest])
        got[:, 5:9] = want[:, 5:9]
        assert torch.equal(got, want)


def test_rows_past_one_pass(w4):
    """More rows than the scratch holds (65536 at R = 128 go in one pass)."""
    import torch
    M = 90000
    y, x, a, b, s = make(6, M, 8, 32, 128, 3)
    ids = np.repeat([0, -1, 2], [70000, 100, M - 70100])
    got = w4.w4_lora(y, x, a, b, dev(ids), scale=s)
    for part in (slice(0, 300), slice(65400, 65700), slice(69990, 70110), slice(89900, 90000)):
        want = w4.w4_lora(y[part].contiguous(), x[part].contiguous(), a, b, dev(ids[part]), scale=s)
        np.testing.assert_allclose(got[part].cpu().numpy(), want.cpu().numpy(), rtol=0, atol=2e-5)
        n = part.stop - part.start
        check(w4, y[part].contiguous(), x[part].contiguous(), a, b, ids[part], s)
    assert torch.equal(got[70000:70100], y[70000:70100])


def test_deterministic_streams_and_graphs(w4):
    """Captured: the adapters of each row are read when the call runs."""
    import torch
    for M in (33, 600):
        y, x, a, b, s = make(7, M, 128, 256, 16, 5)
        sets = [np.random.default_rng(i).integers(-1, 5, M) for i in range(3)]
        want = [w4.w4_lora(y, x, a, b, dev(i), scale=s).clone() for i in sets]
        assert torch.equal(w4.w4_lora(y, x, a, b, dev(sets[0]), scale=s), want[0])
        ids, out = dev(sets[0]), torch.zeros_like(y)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        w4.w4_lora(y, x, a, b, ids, scale=s, out=out, stream=st)
        st.synchronize()
        assert torch.equal(out, want[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            w4.w4_lora(y, x, a, b, ids, scale=s, out=out, stream=st)
            w4.w4_lora(out, x, a, b, ids, scale=s, out=out, stream=st)  # right behind: the scratch is its own again
        for i, w in zip(sets[::-1], want[::-1]):
            twice = w4.w4_lora(w, x, a, b, dev(i), scale=s)
            ids.copy_(dev(i))
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, twice)


def test_binding_checks(w4):
    import torch
    y, x, a, b, s = make(8, 4, 64, 64, 8, 2)
    i = dev([0, 1, 0, -1])
    for bad in (lambda: w4.w4_lora(y.half(), x, a, b, i), lambda: w4.w4_lora(y, x.float(), a, b, i),
                lambda: w4.w4_lora(y, x[:3], a, b, i), lambda: w4.w4_lora(y, x, a, b[:1], i), lambda: w4.w4_lora(y, x, a, b, i[:3]),
                lambda: w4.w4_lora(y, x, a, b, i.long()), lambda: w4.w4_lora(y, x, a, b, i, scale=s[:1]),
                lambda: w4.w4_lora(y, x, a.transpose(1, 2), b, i), lambda: w4.w4_lora(y, x, a, b, i, out=y.bfloat16()),
                lambda: w4.w4_lora(y.t(), x, a, b, i), lambda: w4.w4_lora(y, x, a, b, i, scale=s.double())):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(w4.W4Error):
        w4.w4_lora(y[:, :60].contiguous(), x, a, b[:, :60].contiguous(), i)

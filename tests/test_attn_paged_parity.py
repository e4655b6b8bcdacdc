"""Attention over a paged cache against the fp64 statement (through the public binding).

Elementwise bound, as for the prompt attention (the same arithmetic), times sum_t w_t |v_t|:
  2^-8            each weight rounded to bf16 for the value product
  2^-8            the output rounded to bf16
  2^-15           exp2 of the hardware and the rounding of its argument
  2 D 2^-23 S     the fp32 score sums (S = max of scale * sum_d |q_d k_d|)
  (T/8 + 64) 2^-23  the fp32 accumulation over T keys, the rescales and the merge
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


def dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def f64(t):
    return t.double().cpu().numpy()


class Batch:
    """A pool of pages and sequences over it, every page in a random place."""

    def __init__(self, seed, lq, lens, Hq, Hkv, D, page, layout="rows", spare=2, extra_cols=0):
        import torch
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lq, self.lens = np.array(lq), np.array(lens)
        n = -(-np.maximum(self.lens, 1) // page)
        self.pages, self.page = int(n.sum()) + spare, page
        self.table = np.full((len(lq), int(n.max()) + extra_cols), -1, np.int32)
        order = iter(rng.permutation(self.pages))
        for b in range(len(lq)):
            self.table[b, :n[b]] = [next(order) for _ in range(n[b])]
        self.cu = np.concatenate([[0], np.cumsum(lq)])
        M = max(1, int(self.cu[-1]))
        self.q = torch.randn(M, Hq, D, generator=g, device="cuda").bfloat16()

        def pool(*shape):
            return torch.randn(*shape, generator=g, device="cuda").bfloat16()
        if layout == "rows":
            self.k, self.v = pool(self.pages, page, Hkv, D), pool(self.pages, page, Hkv, D)
        elif layout == "heads":
            self.k, self.v = (pool(self.pages, Hkv, page, D).transpose(1, 2) for _ in range(2))
        elif layout == "inner":  # a row of every page side by side
            self.k, self.v = (pool(page, self.pages, Hkv, D).transpose(0, 1) for _ in range(2))
        else:
            kv = pool(self.pages, 2, page, Hkv, D)
            self.k, self.v = kv[:, 0], kv[:, 1]

    def run(self, w4, window=0, scale=None, step=False, **kw):
        import torch
        scale = self.q.shape[2] ** -0.5 if scale is None else scale
        g = Guard(tuple(self.q.shape), torch.bfloat16)
        g.t.fill_(5.0)
        w4.w4_attn_paged(self.q, self.k, self.v, dev(self.table), dev(self.lens), cu_q=None if step else dev(self.cu),
                         window=window, scale=scale, out=g.t, **kw)
        torch.cuda.synchronize()
        g.check("w4_attn_paged")
        assert w4.device_error() == 0
        return f64(g.t)

    def check(self, w4, window=0, scale=None, step=False):
        D = self.q.shape[2]
        scale = D ** -0.5 if scale is None else scale
        got = self.run(w4, window, scale, step)
        q, k = f64(self.q), f64(self.k)
        ref, ab = serve.attn_paged(q, k, f64(self.v), self.table, self.lens, None if step else self.cu, window, scale)
        S = scale * float(np.sqrt((q ** 2).sum(-1).max() * (k ** 2).sum(-1).max()))
        T = max(1, int(self.lens.max()))
        rel = 2.0 ** -7 + 2.0 ** -15 + 2 * D * 2.0 ** -23 * S + (T / 8 + 64) * 2.0 ** -23
        live = ~np.isnan(ref)
        assert np.isfinite(got[live]).all() and (got[~live] == 5.0).all()
        err, bound = np.abs(got - ref)[live], (rel * ab + 1e-30)[live]
        assert (err <= bound).all(), f"worst ratio {(err / bound).max():.3f}"
        return got


@pytest.mark.parametrize("D", [64, 128, 256, 384, 512])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_widths_and_pages(w4, D, page):
    Batch(D + page, [1, 130, 7, 1], [1, 131, 300, 128], 8, 1, D, page).check(w4)
    Batch(D + page, [33, 1], [700, 513], 4, 2, D, page).check(w4, window=200)
    Batch(D + page, [1, 1, 1, 1, 1], [1, 16, 17, 400, 129], 8, 2, D, page).check(w4, step=True)


@pytest.mark.parametrize("layout", ["heads", "beside", "inner"])
@pytest.mark.parametrize("D,page", [(128, 16), (256, 64), (512, 256)])
def test_layouts_of_the_pool(w4, layout, D, page):
    Batch(3, [40, 1, 3], [300, 90, 3], 6, 2, D, page, layout).check(w4, window=150)
    Batch(4, [1, 1, 1], [300, 90, 3], 6, 2, D, page, layout).check(w4, step=True)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (12, 4), (16, 2), (100, 1), (128, 1)])
def test_head_groups(w4, Hq, Hkv):
    for D in (128, 256):
        Batch(Hq, [20, 1], [150, 40], Hq, Hkv, D, 32).check(w4)
        Batch(Hq, [1, 1, 1], [150, 4, 1000], Hq, Hkv, D, 16).check(w4, step=True)


@pytest.mark.parametrize("step", [False, True])
def test_long_caches_cut_over_many_blocks(w4, step):
    lq = [1, 1] if step else [3, 60]
    Batch(6, lq, [9001, 20000], 4, 1, 128, 16).check(w4, step=step)
    Batch(7, lq, [12000, 77], 8, 1, 512, 64).check(w4, step=step)
    Batch(8, lq, [12000, 8192], 8, 1, 256, 128).check(w4, window=512, step=step)


def test_windows_next_to_edges(w4):
    for w in (1, 2, 16, 127, 128, 129, 512, 2**31 - 1):
        Batch(9, [5, 1], [260, 129], 8, 1, 256, 16).check(w4, window=w)
        Batch(9, [1, 1], [260, 129], 8, 1, 256, 16).check(w4, window=w, step=True)


def test_empty_sequences_lengths_of_zero_and_rows_behind(w4):
    b = Batch(10, [0, 3, 0, 2, 0], [9, 3, 0, 40, 0], 4, 2, 128, 16)
    b.check(w4)
    b = Batch(10, [1, 1, 1], [0, 5, 0], 4, 2, 128, 16)
    got = b.check(w4, step=True)
    assert not got[0].any() and not got[2].any() and got[1].any()
    import torch
    b = Batch(11, [4, 2], [20, 33], 4, 1, 128, 16)
    b.q = torch.cat([b.q, b.q])   # six rows that belong to no sequence
    b.check(w4)
    b = Batch(12, [9, 2], [4, 33], 4, 1, 128, 16)  # more new tokens than positions: the first keep nothing
    got = b.check(w4)
    assert not got[:5].any() and got[5].any()


def test_many_sequences(w4):
    rng = np.random.default_rng(5)
    lq = rng.integers(0, 6, 300)
    lq[100:140] = 0
    Batch(13, lq, lq + rng.integers(0, 140, 300), 2, 1, 128, 16).check(w4)
    Batch(14, np.ones(300, int), rng.integers(0, 300, 300), 4, 1, 64, 32).check(w4, step=True)


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (256, 16), (512, 64), (256, 256)])
def test_absent_pages(w4, D, page):
    """Pages that are none, within and at the ends; a length past the table."""
    for bad in (-1, 10**6, -2**31):
        for step in (False, True):
            b = Batch(15, [1, 1, 1] if step else [4, 60, 1], [600, 450, 70], 8, 2, D, page)
            b.table[0, 0] = b.table[1, 1 if page < 256 else 0] = b.table[2, -(-70 // page) - 1] = bad
            b.check(w4, step=step)
    b = Batch(16, [3, 1], [300, 40], 8, 2, D, page)
    b.table = np.ascontiguousarray(b.table[:, :1])  # the first page alone
    b.check(w4)
    b.table[:] = -1
    assert not b.check(w4).any()


@pytest.mark.parametrize("D,page", [(128, 16), (256, 64), (512, 128), (64, 256)])
@pytest.mark.parametrize("step", [False, True])
def test_nothing_leaks_from_other_rows(w4, D, page, step):
    """NaN and infinities in rows that no sequence holds (behind a length, in spare pages,
    before the window) change nothing; within, they reach the rows that keep them alone."""
    import torch
    window = 90
    b = Batch(17, [1, 1, 1] if step else [50, 3, 1], [250, 70, 17], 8, 2, D, page)
    clean = b.run(w4, window, step=step)
    k0, v0 = b.k.clone(), b.v.clone()
    held = np.zeros((b.pages, page), bool)
    for s, n in enumerate(b.lens):
        for t in range(max(0, n - (b.lq[s] if not step else 1) - window + 1), n):
            held[b.table[s, t // page], t % page] = True
    free = torch.from_numpy(~held).cuda()
    for bad in (float("nan"), float("inf"), float("-inf")):
        b.k, b.v = k0.clone(), v0.clone()
        b.k[free] = bad
        b.v[free] = bad
        np.testing.assert_array_equal(b.run(w4, window, step=step), clean)
    # one value of one key of sequence 0, seen by the rows that keep it
    t = 249 - 45
    for h in range(2):
        b.k, b.v = k0.clone(), v0.clone()
        b.v[b.table[0, t // page], t % page, h, 5] = float("nan")
        got = b.run(w4, window, step=step)
        for m in range(clean.shape[0]):
            pos = 249 if step else 200 + m
            keeps = (m < (1 if step else 50)) and t <= pos and t > pos - window
            row, want = got[m].copy(), clean[m].copy()
            if keeps:
                mine = slice(4 * h, 4 * h + 4)
                assert np.isnan(row[mine, 5]).all()
                row[mine, 5] = want[mine, 5] = 0
            np.testing.assert_array_equal(row, want, err_msg=f"row {m}")


def test_freed_pages_before_the_window_are_not_read(w4):
    b = Batch(18, [3, 1], [500, 200], 8, 1, 256, 16)
    want = b.check(w4, window=100)
    t = b.table.copy()
    b.table[0, :(500 - 3 - 99) // 16] = -7
    b.table[1, :(200 - 100) // 16] = 1 << 29
    np.testing.assert_array_equal(b.run(w4, window=100), want)
    b.table = t


def test_shared_prefix_pages(w4):
    b = Batch(19, [5, 5], [100, 100], 4, 1, 128, 16)
    b.table[1, :5] = b.table[0, :5]
    b.check(w4)


def test_strided_rows(w4):
    import torch
    b = Batch(20, [30, 2], [300, 40], 8, 2, 128, 32)
    want = b.run(w4)
    wide = torch.zeros(32, 8 * 128 + 264, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 1024] = b.q.view(32, 1024)
    ob = torch.full((32, 8 * 128 + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    w4.w4_attn_paged(wide[:, 8:8 + 1024].view(32, 8, 128), b.k, b.v, dev(b.table), dev(b.lens), cu_q=dev(b.cu),
                     scale=128 ** -0.5, out=ob[:, :1024].view(32, 8, 128))
    np.testing.assert_array_equal(f64(ob[:, :1024].reshape(32, 8, 128)), want)
    assert bool((ob[:, 1024:] == 7.0).all())


def test_pool_past_32_bits(w4):
    """Pages whose elements lie past 2^31 in the pool."""
    import torch
    pages, page = 16500, 1024
    k = torch.zeros(pages, page, 1, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = Batch(21, [1, 4], [1500, 1024], 8, 1, 128, page, spare=0)
    far = np.array([pages - 1, 3, pages - 2])
    k[torch.from_numpy(far).cuda()], v[torch.from_numpy(far).cuda()] = small.k, small.v
    for step in (False,):
        want = small.run(w4, step=step)
        small.k, small.v = k, v
        small.table = np.where(small.table >= 0, far[np.maximum(small.table, 0)], -1).astype(np.int32)
        np.testing.assert_array_equal(small.run(w4, step=step), want)
    # a NaN there is found and given to its rows alone (row 400 holds a key in each page)
    v[pages - 1, 400, 0, 3] = float("nan")
    got = small.run(w4)
    assert np.isnan(got[:, :, 3]).any() and np.isfinite(np.delete(got, 3, 2)).all()


@pytest.mark.parametrize("step", [False, True])
def test_deterministic_streams_and_graphs(w4, step):
    """The same bits again, on another stream, and from a captured call whose lengths and
    tables change on the device."""
    import torch
    b = Batch(22, [1, 1, 1] if step else [40, 1, 7], [3000, 64, 500], 8, 1, 256, 16, extra_cols=1)
    want = b.run(w4, step=step)
    np.testing.assert_array_equal(b.run(w4, step=step), want)
    table, lens, cu = dev(b.table), dev(b.lens), None if step else dev(b.cu)
    out = torch.zeros_like(b.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w4.w4_attn_paged(b.q, b.k, b.v, table, lens, cu_q=cu, scale=1 / 16, out=out, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(f64(out), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4_attn_paged(b.q, b.k, b.v, table, lens, cu_q=cu, scale=1 / 16, out=out, stream=s)
    b.lens = np.array([1700, 64, 499])
    b.table = np.ascontiguousarray(b.table[::1])
    b.table[0, :5] = b.table[0, :5][::-1].copy()
    other = b.run(w4, step=step)
    for _ in range(2):
        lens.copy_(dev(b.lens)), table.copy_(dev(b.table))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(f64(out), other)
    assert w4.device_error() == 0


@pytest.mark.parametrize("step", [False, True])
def test_lengths_past_the_table_and_below_zero(w4, step):
    """Positions stay what the length says; the keys end with the table."""
    for D, window in ((128, 0), (256, 0), (512, 0), (128, 70)):
        b = Batch(26, [1, 1, 1, 1], [64, 33, 20, 50], 8, 2, D, 16)
        b.lens = np.array([2**31 - 1, 100, -3, 50])
        b.table[0, 1] = -1
        got = b.check(w4, window=window, step=step)
        assert not got[2].any()
        if window:
            assert not got[0].any()  # its window lies past the table


def test_most_sequences(w4):
    rng = np.random.default_rng(9)
    b = Batch(27, np.ones(4096, int), rng.integers(0, 40, 4096), 1, 1, 64, 16)
    b.check(w4, step=True)
    b.check(w4)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_short_and_long_row_tiles(w4, D):
    """Row tiles that stay whole beside some that are cut, more and fewer of them than blocks."""
    rng = np.random.default_rng(D)
    lq = rng.integers(0, 9, 60)
    lq[7], lq[30], lq[31] = 300, 1, 150
    lens = lq + rng.integers(0, 260, 60)
    Batch(40, lq, lens, 4, 4, D, 16).check(w4)          # all short
    lens[30], lens[31] = 4000, 1700
    Batch(41, lq, lens, 4, 4, D, 16).check(w4)          # two long ones
    Batch(42, lq, lens, 4, 4, D, 64).check(w4, window=300)
    Batch(43, lq[28:33], lens[28:33], 8, 1, D, 32).check(w4)


def test_sharp_and_growing_scores(w4):
    import torch
    for D in (128, 256):
        b = Batch(23, [64, 1], [900, 900], 4, 1, D, 16)
        grow = torch.linspace(0.01, 3.0, 900, device="cuda")
        for s in range(2):
            for p in range(57):
                n = min(16, 900 - 16 * p)
                b.k[b.table[s, p], :n] *= grow[16 * p:16 * p + n, None, None].bfloat16()
        b.check(w4, scale=0.5)
        b = Batch(24, [1, 1], [900, 200], 4, 1, D, 16)
        b.check(w4, scale=1.0, step=True)
    for D in (64, 128, 256, 384, 512):  # the same for single tokens, keys falling as well
        for up in (True, False):
            b = Batch(25, [1, 1, 1], [900, 17, 400], 8, 1, D, 16)
            grow = torch.linspace(0.01, 3.0, 900, device="cuda")
            grow = grow if up else grow.flip(0)
            for s in range(3):
                for p in range(-(-int(b.lens[s]) // 16)):
                    n = min(16, int(b.lens[s]) - 16 * p)
                    b.k[b.table[s, p], :n] *= grow[16 * p:16 * p + n, None, None].bfloat16()
            b.check(w4, scale=0.5, step=True)


def test_short_segments_whole(w4):
    """Windows and tables so short that a block takes whole segments, more and fewer of them than blocks."""
    rng = np.random.default_rng(8)
    for B, D, Hkv, window in ((1, 256, 1, 512), (5, 128, 2, 300), (200, 64, 2, 100), (160, 256, 1, 40), (9, 512, 1, 100)):
        lens = rng.integers(0, 900, B)
        Batch(30 + B, np.ones(B, int), lens, 4 * Hkv, Hkv, D, 16).check(w4, window=window, step=True)
    Batch(29, np.ones(40, int), rng.integers(0, 200, 40), 16, 2, 128, 64).check(w4, step=True)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 3, 1), (64, 16, 1), (128, 16, 2), (256, 8, 1), (256, 11, 1), (384, 6, 2), (512, 8, 1)])
def test_few_short_segments_shared_by_blocks(w4, D, Hq, Hkv):
    """Few sequences on a window or a short table: 2, 4 and 8 blocks have a segment, some of them without a
    tile or without a kept key, and every one's sums are joined."""
    rng = np.random.default_rng(D + Hq)
    for B, keys, window in ((1, 2000, 512), (1, 500, 0), (3, 1000, 300), (3, 300, 0), (9, 260, 0), (9, 900, 200), (20, 700, 257)):
        lens = rng.integers(1, keys + 1, B)
        lens[0] = keys
        if B > 1:
            lens[1], lens[2] = 0, 1
        b = Batch(50 + B, np.ones(B, int), lens, Hq, Hkv, D, 32, extra_cols=1)
        b.check(w4, window=window, step=True)
        n = -(-keys // 32)
        first = max(0, keys - window) // 32 if window else 0
        b.table[0, first + (n - first) // 2:] = -1    # half of the kept keys have no page
        if B > 3:
            b.table[3:5] = b.pages                    # and two sequences none at all
        got = b.check(w4, window=window, step=True)
        assert B <= 3 or not got[3:5].any()


def test_short_segments_one_after_another(w4):
    """Calls of every form of the single tokens in one captured chain, each on the last one's output: a block's
    sums are not written over while another reads them."""
    import torch
    calls = [Batch(60 + i, np.ones(B, int), np.full(B, keys), 8, 1, D, 16)
             for i, (B, keys, D) in enumerate([(3, 512, 256), (1, 512, 256), (3, 5000, 256), (9, 200, 256), (3, 256, 256)])]
    dt = [(dev(b.table), dev(b.lens)) for b in calls]
    outs = [torch.empty_like(b.q) for b in calls]

    def chain(stream=None):
        for i, b in enumerate(calls):
            if i:  # the last output's first row takes the place of a query
                b.q[:1].copy_(outs[i - 1][:1])
            w4.w4_attn_paged(b.q, b.k, b.v, *dt[i], scale=1 / 16, out=outs[i], stream=stream)

    for i, b in enumerate(calls):
        if i:
            b.q[:1].copy_(outs[i - 1][:1])
        w4.w4_attn_paged(b.q, b.k, b.v, *dt[i], scale=1 / 16, out=outs[i])
        torch.cuda.synchronize()
    want = [f64(o) for o in outs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(s)
        s.synchronize()
        for o, x in zip(outs, want):
            np.testing.assert_array_equal(f64(o), x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                chain(s)
        for o in outs:
            o.zero_()
        for _ in range(20):
            g.replay()
        s.synchronize()
    for o, x in zip(outs, want):
        np.testing.assert_array_equal(f64(o), x)
    assert w4.device_error() == 0


def test_binding_checks(w4):
    import torch
    q = torch.zeros(4, 8, 256, dtype=torch.bfloat16, device="cuda")
    p = torch.zeros(4, 16, 1, 256, dtype=torch.bfloat16, device="cuda")
    t, n, cu = dev([[0], [1]]), dev([3, 4]), dev([0, 2, 4])
    for bad in (lambda: w4.w4_attn_paged(q.float(), p, p, t, n, cu), lambda: w4.w4_attn_paged(q, p, p[:2], t, n, cu),
                lambda: w4.w4_attn_paged(q, p, p, t.long(), n, cu), lambda: w4.w4_attn_paged(q, p, p, t, n[:1], cu),
                lambda: w4.w4_attn_paged(q, p, p, t, n, cu[:2]), lambda: w4.w4_attn_paged(q, p, p, t, n),
                lambda: w4.w4_attn_paged(q, p.float(), p.float(), t, n, cu), lambda: w4.w4_attn_paged(q, p[..., ::2], p[..., ::2], t, n, cu),
                lambda: w4.w4_attn_paged(q, p, p, t[0], n, cu), lambda: w4.w4_attn_paged(q, p, p, t, n, cu, out=q[:3])):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for kw in (dict(scale=0.0), dict(window=-1)):
        with pytest.raises(w4.W4Error):
            w4.w4_attn_paged(q, p, p, t, n, cu, **kw)
    with pytest.raises(w4.W4Error):
        w4.w4_attn_paged(q, p[:, :8], p[:, :8], t, n, cu)

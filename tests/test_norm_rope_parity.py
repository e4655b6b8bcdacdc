"""Norms with rotation and the paged store against the fp64 statement.

Elementwise bound, derived from the kernel's arithmetic, for an element of a turned pair
(a, b) with size = |a| + |b| (|u| where nothing is turned):
  2^-8 |out|     the output rounded to bf16 (half a step), doubled neither way
  size 2^-19     fp32: the mean square over D <= 512 elements (at most 24 roundings deep in
                 lanes, halved by the root), rsqrtf (2^-22) and two products: 18 2^-24; the
                 angle rounded to fp32 below pi: 3.2 2^-24; sine and cosine (1 ulp): 2 2^-24;
                 two products and a sum: 2 2^-24. Together 26 2^-24 < 2^-19.
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


def close(got, u, pos, f, pairs, what=""):
    ref, size = serve.turn(u, pos, f, pairs)
    err = np.abs(got - ref)
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * (1 + 2.0 ** -8) * size + 1e-38
    assert np.isfinite(got).all() and (err <= bound).all(), f"{what}: worst {(err / bound).max():.3f}"


def freqs(R, base=1e4):
    return (base ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)


def f64(t):
    return t.double().cpu().numpy()


def dev(a, dt=np.int32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()


def rows(M, Hq, Hkv, D, seed, dtype, extra=0):
    """q, k, v as views of one fused projection."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    y = (torch.randn(M, (Hq + 2 * Hkv) * D + extra, generator=g, device="cuda") * 3).to(dtype)
    return (y[:, :Hq * D].view(M, Hq, D), y[:, Hq * D:(Hq + Hkv) * D].view(M, Hkv, D),
            y[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(M, Hkv, D))


def weight(D, seed):
    import torch
    return 1 + 0.3 * torch.randn(D, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (128, 128), (128, 8), (256, 256), (256, 64), (384, 384), (384, 96),
                                 (512, 512), (512, 128), (256, 0)])
def test_widths_and_styles(w4, D, R, pairs, dtype):
    import torch
    for M, Hq, Hkv in ((1, 8, 1), (37, 6, 2), (2, 1, 1)):
        q, k, _ = rows(M, Hq, Hkv, D, D + R, getattr(torch, dtype))
        qw, kw, f = weight(D, 1), weight(D, 2), freqs(R)
        pos = np.random.default_rng(3).integers(0, 131072, M).astype(np.int32)
        gq, gk = Guard((M, Hq, D), torch.bfloat16), Guard((M, Hkv, D), torch.bfloat16)
        w4.w4_qk_norm_rope(q, k, dev(pos), dev(f, np.float32) if R else None, q_weight=qw, k_weight=kw, pairs=pairs,
                           q_out=gq.t, k_out=gk.t)
        torch.cuda.synchronize()
        gq.check("q"), gk.check("k")
        close(f64(gq.t), serve.norm(f64(q), f64(qw), 1e-6), pos, f, pairs, "q")
        close(f64(gk.t), serve.norm(f64(k), f64(kw), 1e-6), pos, f, pairs, "k")


@pytest.mark.parametrize("M,Hq,Hkv,D", [(5000, 8, 1, 64), (700, 16, 2, 384), (3, 100, 100, 128)])
def test_many_rows_and_heads(w4, M, Hq, Hkv, D):
    import torch
    q, k, _ = rows(M, Hq, Hkv, D, 9, torch.float32)
    pos = np.arange(M, dtype=np.int32) + 1000
    qo, ko = w4.w4_qk_norm_rope(q, k, dev(pos), dev(freqs(D), np.float32), q_weight=weight(D, 5))
    close(f64(qo), serve.norm(f64(q), f64(weight(D, 5)), 1e-6), pos, freqs(D), False, "q")
    close(f64(ko), f64(k), pos, freqs(D), False, "k")  # no weight: turned alone


def test_far_positions_and_odd_frequencies(w4):
    """Positions to both ends of 32 bits; frequencies of zero, below zero, above a turn, tiny and subnormal."""
    import torch
    pos = np.array([0, 1, -1, 131071, 2**24 + 1, 2**31 - 1, -2**31, 123456789], np.int32)
    f = np.concatenate([freqs(96), [0.0, -0.3, 7.0, 100000.25, 2e-12, 1e-30, 1e-45, 2.0**23 + 1],
                        freqs(48, 1e6)]).astype(np.float32)
    q, k, _ = rows(len(pos), 4, 1, 256, 21, torch.float32)
    assert len(f) == 80
    for pairs in (False, True):
        qo, ko = w4.w4_qk_norm_rope(q, k, dev(pos), dev(f, np.float32), pairs=pairs)
        close(f64(qo), f64(q), pos, f, pairs, "q")
        close(f64(ko), f64(k), pos, f, pairs, "k")


def test_queries_alone_in_place_and_zero_heads(w4):
    import torch
    q, _, _ = rows(9, 8, 1, 128, 4, torch.bfloat16)
    w, f, pos = weight(128, 3), freqs(128), np.arange(9, dtype=np.int32)
    want, none = w4.w4_qk_norm_rope(q, None, dev(pos), dev(f, np.float32), q_weight=w)
    assert none is None
    mine = q.clone()
    w4.w4_qk_norm_rope(mine, None, dev(pos), dev(f, np.float32), q_weight=w, q_out=mine)
    assert torch.equal(mine, want)
    z = torch.zeros(2, 3, 128, device="cuda")
    out, _ = w4.w4_qk_norm_rope(z, z, dev([5, 6]), dev(f, np.float32), q_weight=w, k_weight=w)
    assert not out.any()  # eps keeps a head of zeros zero
    big = torch.full((1, 1, 128), 1e18, device="cuda")
    out, _ = w4.w4_qk_norm_rope(big, None, dev([0]), None, q_weight=torch.ones(128, device="cuda"), eps=0.0)
    assert torch.equal(out, torch.ones_like(out))


def test_nan_stays_in_its_head(w4):
    import torch
    for D in (64, 256, 512):
        q, k, _ = rows(4, 3, 2, D, 6, torch.float32)
        w, f, pos = weight(D, 3), dev(freqs(D), np.float32), dev([3, 4, 5, 6])
        a, b = w4.w4_qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w)
        q[1, 2, 7] = float("nan")
        c, d = w4.w4_qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w)
        assert torch.isnan(c[1, 2]).all() and torch.equal(b, d)
        c[1, 2] = a[1, 2]
        assert torch.equal(a, c)


# ------------------------------------------------------------------- to pages

def store(w4, seed, lq, past, Hq, Hkv, D, R, page, dtype="float32", layout="rows", norm_v=True, spare=2, rows_behind=0,
          step=False, table=None, status=False):
    """Runs w4_qkv_paged and compares q_out, every page and the status with the statement."""
    import torch
    rng = np.random.default_rng(seed)
    lens = np.array(lq) + np.array(past)
    M = sum(lq) + rows_behind
    n = -(-np.maximum(lens, 1) // page)
    pages = int(n.sum()) + spare
    if table is None:
        order = iter(rng.permutation(pages))
        table = np.full((len(lq), int(n.max())), -1, np.int32)
        for b in range(len(lq)):
            table[b, :n[b]] = [next(order) for _ in range(n[b])]
    cu = np.concatenate([[0], np.cumsum(lq)])
    q, k, v = rows(M, Hq, Hkv, D, seed, getattr(torch, dtype))
    qw, kw, vw, f = weight(D, 1), weight(D, 2), weight(D, 4) if norm_v else None, freqs(R)
    if layout == "rows":
        g = [Guard((pages, page, Hkv, D), torch.bfloat16) for _ in range(2)]
        kp, vp = g[0].t, g[1].t
    elif layout == "heads":
        g = [Guard((pages, Hkv, page, D), torch.bfloat16) for _ in range(2)]
        kp, vp = (x.t.transpose(1, 2) for x in g)
    elif layout == "inner":  # a row of every page side by side
        g = [Guard((page, pages, Hkv, D), torch.bfloat16) for _ in range(2)]
        kp, vp = (x.t.transpose(0, 1) for x in g)
    else:  # keys and values of a page side by side
        g = [Guard((pages, 2, page, Hkv, D), torch.bfloat16)]
        kp, vp = g[0].t[:, 0], g[0].t[:, 1]
    for x in g:
        x.t.fill_(9.0)
    out = Guard((M, Hq, D), torch.bfloat16)
    out.t.fill_(5.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status else None
    w4.w4_qkv_paged(q, k, v, kp, vp, dev(table), dev(lens), dev(f, np.float32) if R else None,
                    cu_q=None if step else dev(cu), q_weight=qw, k_weight=kw, v_weight=vw, q_out=out.t, status=st)
    torch.cuda.synchronize()
    out.check("q_out")
    for x in g:
        x.check("pages")
    seq, pos = serve.rows_of(None if step else cu, lens, M)
    live = seq >= 0
    close(f64(out.t)[live], serve.norm(f64(q), f64(qw), 1e-6)[live], pos[live], f, False, "q")
    assert (f64(out.t)[~live] == 5.0).all()
    kn, vn = serve.norm(f64(k), f64(kw), 1e-6), serve.norm(f64(v), None if vw is None else f64(vw), 1e-6)
    gk, gv = f64(kp), f64(vp)
    left = np.ones(gk.shape[:2], bool)
    lost = 0
    for m in np.flatnonzero(live):
        at = serve.place(table, pages, page, seq[m], pos[m])
        if at is None:
            lost = 1
            continue
        left[at] = False
        close(gk[at][None], kn[m:m + 1], pos[m:m + 1], f, False, f"key {m}")
        close(gv[at][None], vn[m:m + 1], [0], None, False, f"value {m}")
    assert (gk[left] == 9.0).all() and (gv[left] == 9.0).all()
    if status:
        assert int(st) == lost
    return lost


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("layout", ["rows", "heads", "beside", "inner"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_store_layouts(w4, page, layout, dtype):
    store(w4, 1, [1, 40, 3, 17], [0, 5, 1000, 15], 8, 2, 128, 128, page, dtype, layout, status=True)
    store(w4, 2, [1, 1, 1], [0, 15, 16], 3, 1, 512, 256, page, dtype, layout, norm_v=False, step=True, status=True)


def test_store_empty_sequences_and_rows_behind(w4):
    store(w4, 3, [0, 4, 0, 0, 2, 0], [7, 0, 0, 30, 5, 0], 2, 1, 64, 64, 16, rows_behind=9, status=True)
    store(w4, 4, [1], [0], 3, 3, 384, 384, 32, rows_behind=1, status=True)


def test_store_without_a_page(w4):
    """Absent pages and positions past the table or below zero are not stored and set the status."""
    t = np.array([[-1, 3], [7, 2], [1, 400]], np.int32)
    assert store(w4, 5, [4, 3, 5], [10, 30, 16], 2, 1, 128, 128, 16, spare=2, table=t, status=True) == 1
    assert store(w4, 6, [4], [15], 2, 1, 128, 128, 16, spare=3, table=np.array([[2, 0]], np.int32), status=True) == 0
    import torch
    q, k, v = rows(5, 2, 1, 128, 8, torch.float32)
    kp = torch.full((2, 16, 1, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    vp, st = kp.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    # five rows of a sequence of length 3: positions -2 .. 2
    w4.w4_qkv_paged(q, k, v, kp, vp, dev([[1]]), dev([3]), None, cu_q=dev([0, 5]), status=st)
    assert int(st) == 1 and bool((kp[0] == 9).all()) and bool((kp[1, 3:] == 9).all())
    assert torch.equal(vp[1, :3], v[2:].bfloat16())


def test_store_lengths_at_the_ends(w4):
    """Lengths of 2^31 - 1 and below zero; 4096 sequences, some empty."""
    import torch
    q, k, v = rows(2, 2, 1, 128, 8, torch.float32)
    kp = torch.full((2, 16, 1, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    vp, st = kp.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    f = freqs(128)
    got = w4.w4_qkv_paged(q, k, v, kp, vp, dev([[0], [1]]), dev([2**31 - 1, -7]), dev(f, np.float32), status=st)
    assert int(st) == 1 and bool((kp == 9).all()) and bool((vp == 9).all())
    close(f64(got), f64(q), np.array([2**31 - 2, -1]), f, False)
    rng = np.random.default_rng(3)
    lq = rng.integers(0, 3, 4096)
    store(w4, 7, lq.tolist(), rng.integers(0, 30, 4096).tolist(), 1, 1, 64, 64, 16, status=True)


def test_store_far_in_a_large_pool(w4):
    """Elements past 2^31 of the pool."""
    import torch
    pages = 16500
    kp = torch.zeros(pages, 1024, 1, 128, dtype=torch.bfloat16, device="cuda")  # 2.16e9 elements
    vp = torch.zeros_like(kp)
    q, k, v = rows(2, 2, 1, 128, 8, torch.float32)
    w4.w4_qkv_paged(q, k, v, kp, vp, dev([[pages - 1], [0]]), dev([1024, 1]), None, q_weight=weight(128, 1))
    assert torch.equal(vp[pages - 1, 1023], v[0].bfloat16()) and torch.equal(kp[0, 0], k[1].bfloat16())
    assert int((vp[1:pages - 1].view(torch.int16) != 0).sum()) == 0


def test_graph_and_stream(w4):
    """A captured call serves every step: lengths and tables are read when it runs."""
    import torch
    q, k, v = rows(3, 8, 1, 256, 8, torch.float32)
    kp = torch.zeros(6, 16, 1, 256, dtype=torch.bfloat16, device="cuda")
    vp, f = torch.zeros_like(kp), dev(freqs(256), np.float32)
    table, lens = dev([[0, 1], [2, 3], [4, 5]]), dev([1, 16, 30])
    w = weight(256, 2)
    out = torch.zeros(3, 8, 256, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4_qkv_paged(q, k, v, kp, vp, table, lens, f, k_weight=w, q_out=out, stream=s)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        k2, v2 = torch.zeros_like(kp), torch.zeros_like(vp)
        q2 = w4.w4_qkv_paged(q, k, v, k2, v2, table, lens, f, k_weight=w)
        assert torch.equal(q2, out)
        for b, n in enumerate(lens.tolist()):
            pg = table[b, (n - 1) // 16], (n - 1) % 16
            assert torch.equal(kp[pg], k2[pg]) and torch.equal(vp[pg], v2[pg]) and bool(kp[pg].any())
        lens += 1


def test_binding_checks(w4):
    import torch
    q, k, v = rows(3, 8, 2, 128, 8, torch.float32)
    f, pos = dev(freqs(128), np.float32), dev([1, 2, 3])
    kp = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    t, n = dev([[0], [1], [2]]), dev([1, 1, 1])
    for bad in (lambda: w4.w4_qk_norm_rope(q, k.bfloat16(), pos, f), lambda: w4.w4_qk_norm_rope(q.half(), k, pos, f),
                lambda: w4.w4_qk_norm_rope(q, k, pos.long(), f), lambda: w4.w4_qk_norm_rope(q, k, pos[:2], f),
                lambda: w4.w4_qk_norm_rope(q, k, pos, f.double()), lambda: w4.w4_qk_norm_rope(q, k[:2], pos, f),
                lambda: w4.w4_qk_norm_rope(q, k, pos, f, q_weight=f), lambda: w4.w4_qk_norm_rope(q, k, pos, f, q_out=q),
                lambda: w4.w4_qk_norm_rope(q.transpose(0, 1), None, pos, f),
                lambda: w4.w4_qkv_paged(q, k, v, kp, kp.float(), t, n, f), lambda: w4.w4_qkv_paged(q, k, v, kp, kp[:3], t, n, f),
                lambda: w4.w4_qkv_paged(q, k, v, kp, kp.transpose(1, 2).contiguous().transpose(1, 2), t, n, f),
                lambda: w4.w4_qkv_paged(q, k, v, kp, kp, t[:2], n[:2], f), lambda: w4.w4_qkv_paged(q, k, v, kp, kp, t, n[:2], f),
                lambda: w4.w4_qkv_paged(q, k, v, kp, kp, t, n, f, cu_q=n), lambda: w4.w4_qkv_paged(q, k, v, kp, kp, t.long(), n, f)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(w4.W4Error):
        w4.w4_qk_norm_rope(q, k, pos, f, eps=-1.0)
    with pytest.raises(w4.W4Error):
        w4.w4_qk_norm_rope(q, k, pos, f[:33])

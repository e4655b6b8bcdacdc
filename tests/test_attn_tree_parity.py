"""Attention of drafted trees over a cache against the fp64 statement; the bound is
that of the prompt attention (the same arithmetic)."""
import numpy as np
import pytest

import synth
from _guard import Guard
from oracle import draft
from test_attn_prompt_parity import rel_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import bit_weight_only_w4a16_gb300 as w4
    w4.init()
    return w4


def random_tree(rng, N):
    p = np.full(N, -1, np.int32)
    for i in range(1, N):
        p[i] = rng.integers(max(-1, i - 6), i)
    return p


def make(seed, B, N, T, Hq, Hkv, D):
    import torch
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).bfloat16() for s in
            ((B, N, Hq, D), (B, T, Hkv, D), (B, T, Hkv, D), (B, N, Hkv, D), (B, N, Hkv, D))]


def run(w4, q, k, v, kt, vt, parents, pos, kpos, window, scale, **kw):
    import torch
    g = Guard(tuple(q.shape), torch.bfloat16)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()

    w4.w4_attn_tree(*(x.cuda() for x in (q, k, v, kt, vt)), dev(parents), dev(pos),
                    kpos=None if kpos is None else dev(kpos), window=window, scale=scale, out=g.t, **kw)
    torch.cuda.synchronize()
    g.check("w4_attn_tree")
    assert w4.device_error() == 0
    return g.t.float().cpu().numpy().astype(np.float64)


def check(w4, seed, B, N, T, Hq, Hkv, D, parents, pos, kpos=None, window=0, poison=True):
    """Slots that no node keeps hold NaN."""
    t = make(seed, B, N, T, Hq, Hkv, D)
    scale = D ** -0.5
    f = [x.float().numpy().astype(np.float64) for x in t]
    ref, ab = draft.attn_tree(*f, parents, pos, kpos, window, scale)
    if poison:
        for b in range(B):
            kept = draft.tree_keep(parents[b], pos[b], None if kpos is None else kpos[b], T, window)[:, :T].any(0)
            t[1][b][~kept] = float("nan")
            t[2][b][~kept] = float("nan")
    got = run(w4, *t, parents, pos, kpos, window, scale)
    S = scale * float(np.sqrt((f[0] ** 2).sum(-1).max() * max((f[1] ** 2).sum(-1).max(), (f[3] ** 2).sum(-1).max())))
    assert np.isfinite(got).all()
    err, bound = np.abs(got - ref), rel_bound(D, S, T + N) * ab + 1e-30
    assert (err <= bound).all(), f"worst ratio {(err / bound).max():.3f}"
    return got


@pytest.mark.parametrize("D", [64, 128, 256, 384, 512])
@pytest.mark.parametrize("N,T,pos", [(1, 1, 1), (8, 300, 257), (17, 1000, 128), (64, 130, 130), (5, 64, 0)])
def test_full_cache(w4, D, N, T, pos):
    rng = np.random.default_rng(N)
    check(w4, D + N, 1, N, T, 8, 1, D, random_tree(rng, N)[None], [pos])


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (4, 4), (12, 4), (128, 1)])
def test_head_groups_and_batches(w4, Hq, Hkv):
    rng = np.random.default_rng(Hq)
    B, N, T = 3, 9, 400
    check(w4, Hq, B, N, T, Hq, Hkv, 128, np.stack([random_tree(rng, N) for _ in range(B)]), [400, 1, 129])


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("T,pos,window", [(512, 1300, 512), (512, 100, 512), (200, 777, 200), (300, 299, 40), (96, 5, 3)])
def test_rings_with_windows(w4, D, T, pos, window):
    """A ring as long as its window (or longer), full and partly empty; a chain of
    nodes, so that the windows of deeper nodes begin later."""
    N = 12
    chain = np.arange(-1, N - 1, dtype=np.int32)
    kpos = synth.ring_positions(pos - 1, T)[None]
    check(w4, T + pos, 1, N, T, 8, 1, D, chain[None], [pos], kpos, window)
    check(w4, T + pos + 1, 1, N, T, 8, 1, D, random_tree(np.random.default_rng(1), N)[None], [pos], kpos, 0)


@pytest.mark.parametrize("window", [1, 5, 100])
def test_window_on_a_full_cache(w4, window):
    N = 20
    chain = np.arange(-1, N - 1, dtype=np.int32)
    check(w4, window, 1, N, 700, 8, 2, 128, chain[None], [613], None, window)


def test_scattered_slot_table(w4):
    """Positions in any order, some empty, some not committed yet."""
    rng = np.random.default_rng(3)
    T = 333
    kpos = rng.permutation(2 * T)[:T].astype(np.int32)
    kpos[rng.random(T) < 0.2] = -1
    check(w4, 4, 1, 10, T, 8, 1, 256, random_tree(rng, 10)[None], [400], kpos[None], 150)


@pytest.mark.parametrize("D", [128, 512])
def test_absent_nodes_and_odd_parents(w4, D):
    """-2 gives zeros; a parent at or after its node, or below -2, counts as none."""
    parents = np.array([[-1, 0, -2, 1, 4, -7, 63, 3]], np.int32)
    got = check(w4, 6, 1, 8, 200, 8, 1, D, parents, [150])
    assert not got[0, 2].any() and got[0, 3].any()


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_siblings_do_not_leak(w4, D):
    """NaN and infinities in a node reach its descendants and itself alone."""
    N, T = 9, 140
    parents = np.array([[-1, 0, 0, 1, 2, 3, 4, 2, 0]], np.int32)
    t = make(7, 1, N, T, 8, 1, D)
    clean = run(w4, *t, parents, [T], None, 0, D ** -0.5)
    for val in (float("nan"), float("inf")):
        for i, x in ((3, "k"), (4, "v")):
            t2 = [y.clone() for y in t]
            t2[i][0, 2] = val
            got = run(w4, *t2, parents, [T], None, 0, D ** -0.5)
            for n in range(N):
                if 2 not in draft.tree_chain(parents[0], n):
                    np.testing.assert_array_equal(got[0, n], clean[0, n])
                elif x == "v" or np.isnan(val):
                    assert not np.isfinite(got[0, n]).any()


@pytest.mark.parametrize("D", [64, 256, 512])
def test_windowed_slots_do_not_leak(w4, D):
    """A slot that the first level's window still reaches and deeper nodes' do not."""
    N, T, pos, window = 6, 128, 500, 100
    chain = np.arange(-1, N - 1, dtype=np.int32)[None]
    for kpos in (None, synth.ring_positions(pos - 1, T)[None]):
        TT = T if kpos is not None else pos
        t = make(8, 1, N, TT, 4, 1, D)
        clean = run(w4, *t, chain, [pos], kpos, window, 0.1)
        p = pos - window + 3  # kept by depths 0 .. 2
        slot = p if kpos is None else int(np.flatnonzero(kpos[0] == p)[0])
        t[2][0, slot] = float("nan")
        got = run(w4, *t, chain, [pos], kpos, window, 0.1)
        for n in range(N):
            if n <= 2:
                assert not np.isfinite(got[0, n]).any()
            else:
                np.testing.assert_array_equal(got[0, n], clean[0, n])


def test_one_node_is_decode_attention(w4):
    """N = 1 against the decode attention: the query at pos, its own key appended."""
    import torch
    H, T, D, pos = 8, 900, 256, 700
    q, k, v, kt, vt = (x.cuda() for x in make(9, 1, 1, T, H, 1, D))
    one = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    got = w4.w4_attn_tree(q, k, v, kt, vt, one([[-1]]), one([pos]), scale=D ** -0.5)
    kc, vc = k[0, :, 0].clone(), v[0, :, 0].clone()
    kc[pos], vc[pos] = kt[0, 0, 0], vt[0, 0, 0]
    want = w4.w4_attn_decode(q[0, 0].contiguous(), kc, vc, qpos=pos, scale=D ** -0.5)
    # both round fp32 sums; the tree also its weights and its output to bf16
    assert (got[0, 0].float() - want).abs().max().item() <= 2.0 ** -7 * v.float().abs().max().item()


def test_cache_past_32_bit_offsets(w4):
    """2^31 elements and more in a cache: the kept slots lie behind them."""
    import torch
    D, N = 512, 4
    T = (1 << 22) + 200
    kc = torch.zeros(1, T, 1, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros(1, T, 1, D, dtype=torch.bfloat16, device="cuda")
    q, k, v, kt, vt = make(11, 1, N, 300, 8, 1, D)
    kc[0, -300:], vc[0, -300:] = k[0].cuda(), v[0].cuda()
    parents = np.array([[-1, 0, 1, 0]], np.int32)
    window = 250
    got = run(w4, q, kc, vc, kt, vt, parents, [T], None, window, D ** -0.5)
    f = [x.float().numpy().astype(np.float64) for x in (q, k, v, kt, vt)]
    ref, ab = draft.attn_tree(*f, parents, [300], None, window, D ** -0.5)
    S = D ** -0.5 * float(np.sqrt((f[0] ** 2).sum(-1).max() * (f[1] ** 2).sum(-1).max()))
    assert (np.abs(got - ref) <= rel_bound(D, S, 300) * ab).all()


def test_device_positions_in_a_graph(w4):
    """One captured call serves every step: pos and parents change on the device."""
    import torch
    N, T, D = 8, 1024, 256
    t = [x.cuda() for x in make(12, 1, N, T, 8, 1, D)]
    steps = [(5, np.arange(-1, N - 1)), (1000, random_tree(np.random.default_rng(2), N)), (0, np.full(N, -1))]
    want = [run(w4, *(x.cpu() for x in t), p[None].astype(np.int32), [pos], None, 0, 0.1) for pos, p in steps]
    par, pos = torch.zeros(1, N, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, s = torch.empty_like(t[0]), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4_attn_tree(*t, par, pos, scale=0.1, out=out, stream=s)
    for (ps, p), w in zip(steps, want):
        par.copy_(torch.from_numpy(p[None].astype(np.int32)))
        pos.fill_(ps)
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(out.double().cpu().numpy(), w)

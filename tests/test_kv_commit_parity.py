"""Accepted paths stored into caches and rings: bit-exact."""
import numpy as np
import pytest

import synth
from _guard import Guard
from oracle import draft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import bit_weight_only_w4a16_gb300 as w4
    w4.init()
    return w4


def check(w4, seed, L, B, T, N, W, path, count, pos, ring):
    import torch
    rng = np.random.default_rng(seed)
    kc, vc = (rng.integers(0, 1 << 15, (L, B, T, W)).astype(np.int16) for _ in range(2))
    kt, vt = (rng.integers(0, 1 << 15, (L, B, N, W)).astype(np.int16) for _ in range(2))
    kpos = np.stack([synth.ring_positions(p - 1, T) for p in pos]) if ring else None
    gk, gv = Guard(kc.shape, torch.int16), Guard(vc.shape, torch.int16)
    gk.t.copy_(torch.from_numpy(kc)), gv.t.copy_(torch.from_numpy(vc))
    gp = None
    if ring:
        gp = Guard(kpos.shape, torch.int32)
        gp.t.copy_(torch.from_numpy(kpos))

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()

    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = dev(pos)
    w4.w4_kv_commit(gk.t, gv.t, torch.from_numpy(kt).cuda(), torch.from_numpy(vt).cuda(), dev(path), dev(count), p,
                    kpos=None if gp is None else gp.t, status=st)
    torch.cuda.synchronize()
    for g in (gk, gv, gp):
        if g is not None:
            g.check("w4_kv_commit")
    rk, rv, rp, rs = draft.kv_commit(kc, vc, kpos, kt, vt, path, count, pos)
    np.testing.assert_array_equal(gk.t.cpu().numpy(), rk)
    np.testing.assert_array_equal(gv.t.cpu().numpy(), rv)
    if ring:
        np.testing.assert_array_equal(gp.t.cpu().numpy(), rp)
    assert int(st.item()) == rs and p.cpu().numpy().tolist() == list(pos)
    return rs


@pytest.mark.parametrize("L,B,W", [(1, 1, 8), (3, 2, 256), (28, 1, 512), (2, 5, 1032)])
@pytest.mark.parametrize("ring", [False, True])
def test_paths(w4, L, B, W, ring):
    rng = np.random.default_rng(L + W)
    N, T = 17, 64
    path = np.stack([np.sort(rng.choice(N, N, replace=False)) for _ in range(B)])
    count = rng.integers(0, N + 1, B)
    pos = rng.integers(0, T - N, B) if not ring else rng.integers(0, 1000, B)
    assert check(w4, 1, L, B, T, N, W, path, count, pos.tolist(), ring) == 0


def test_wrap_and_short_ring(w4):
    path = np.arange(9)[None]
    assert check(w4, 2, 2, 1, 16, 9, 64, path, [9], [13], True) == 0       # wraps past slot 15
    assert check(w4, 3, 2, 1, 4, 9, 64, path, [9], [6], True) == 0         # the last four stay
    assert check(w4, 4, 1, 1, 1, 9, 64, path, [9], [0], True) == 0


@pytest.mark.parametrize("count", [-3, 0, 5, 8, 100])
def test_counts_are_cut(w4, count):
    check(w4, 5, 2, 1, 32, 8, 64, np.arange(8)[None], [count], [3], False)


def test_refused_entries_are_skipped(w4):
    assert check(w4, 6, 2, 1, 8, 4, 64, [[0, -1, 4, 3]], [4], [2], False) == 1   # nodes
    assert check(w4, 7, 2, 1, 8, 4, 64, [[0, 1, 2, 3]], [4], [6], False) == 1    # past a full cache
    assert check(w4, 8, 2, 2, 8, 4, 64, [[0, 1, 2, 3], [3, 3, 3, 3]], [4, 2], [-2, 1], False) == 1


def test_refusals(w4):
    import torch
    c = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: w4.w4_kv_commit(c, c[:, :, :8], t, t, i, i[:1], i[:1]),
                lambda: w4.w4_kv_commit(c, c, t, t, i[:3], i[:1], i[:1]),
                lambda: w4.w4_kv_commit(c.float(), c, t, t, i, i[:1], i[:1]),
                lambda: w4.w4_kv_commit(c, c, t, t, i, i[:1], i[:1], kpos=i)):
        with pytest.raises((TypeError, ValueError)):
            bad()

"""Prompt attention against the fp64 statement (through the public binding).

Elementwise bound, derived from the kernel's arithmetic, times sum_t w_t |v_t|:
  2^-8            each weight rounded to bf16 for the value product (bf16 has 8
                  significant bits: 1 + 2^-8 lies half-way between 1 and 1 + 2^-7)
  2^-8            the output rounded to bf16
  2^-15           exp2 of the hardware and the rounding of its argument
  2 D 2^-23 S     the fp32 score sums (S = max of scale * sum_d |q_d k_d|)
  (T/8 + 64) 2^-23  the fp32 accumulation over T keys, the rescales and the merge
"""
import numpy as np
import pytest

from _guard import Guard
from oracle import draft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import bit_weight_only_w4a16_gb300 as w4
    w4.init()
    return w4


def rel_bound(D, S, T):
    return 2.0 ** -7 + 2.0 ** -15 + 2 * D * 2.0 ** -23 * S + (T / 8 + 64) * 2.0 ** -23


def make(seed, lq, lk, Hq, Hkv, D):
    import torch
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(max(sum(lq), 1), Hq, D, generator=g).bfloat16()
    k = torch.randn(max(sum(lk), 1), Hkv, D, generator=g).bfloat16()
    v = torch.randn(max(sum(lk), 1), Hkv, D, generator=g).bfloat16()
    cu_q = np.concatenate([[0], np.cumsum(lq)]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum(lk)]).astype(np.int32)
    return q, k, v, cu_q, cu_k


def run(w4, q, k, v, cu_q, cu_k, window, scale, **kw):
    import torch
    g = Guard(tuple(q.shape), torch.bfloat16)
    cq = torch.from_numpy(cu_q).cuda()
    ck = None if cu_k is None else torch.from_numpy(cu_k).cuda()
    w4.w4_attn_prompt(q.cuda() if not q.is_cuda else q, k.cuda() if not k.is_cuda else k,
                      v.cuda() if not v.is_cuda else v, cq, ck, window=window, scale=scale, out=g.t, **kw)
    torch.cuda.synchronize()
    g.check("w4_attn_prompt")
    assert w4.device_error() == 0
    return g.t.float().cpu().numpy().astype(np.float64)


def check(w4, seed, lq, lk, Hq, Hkv, D, window=0, scale=None):
    q, k, v, cu_q, cu_k = make(seed, lq, lk, Hq, Hkv, D)
    scale = D ** -0.5 if scale is None else scale
    got = run(w4, q, k, v, cu_q, cu_k, window, scale)
    qf, kf, vf = (x.float().numpy().astype(np.float64) for x in (q, k, v))
    ref, ab = draft.attn_prompt(qf, kf, vf, cu_q, cu_k, window, scale)
    S = scale * float(np.abs(qf).sum(-1).max() * np.abs(kf).max())
    S = min(S, scale * float(np.sqrt((qf ** 2).sum(-1).max() * (kf ** 2).sum(-1).max())))
    n = sum(lq)
    err, bound = np.abs(got - ref)[:n], (rel_bound(D, S, max(max(lk), 1)) * ab + 1e-30)[:n]
    assert np.isfinite(got[:n]).all()
    assert (err <= bound).all(), f"worst ratio {(err / bound).max():.3f}"
    return got, ref


@pytest.mark.parametrize("D", [64, 128, 256, 384, 512])
@pytest.mark.parametrize("lq,window", [([1], 0), ([127, 1, 2, 130], 0), ([300], 100), ([65, 64], 1)])
def test_lengths_and_windows(w4, D, lq, window):
    check(w4, 10 + D, lq, lq, 8, 1, D, window)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (4, 4), (12, 4), (7, 1), (16, 2), (48, 1), (100, 1), (128, 1)])
@pytest.mark.parametrize("D", [128, 256])
def test_head_groups(w4, Hq, Hkv, D):
    check(w4, 20 + Hq, [40, 5], [133, 5], Hq, Hkv, D)


@pytest.mark.parametrize("D", [64, 256, 512])
def test_chunks_of_longer_prompts(w4, D):
    """More keys than queries, cut over many SMs; lengths off the tiles."""
    check(w4, 30, [5, 33, 1], [1500, 129, 4001], 4, 2, D)
    check(w4, 31, [17], [2049], 8, 1, D, window=700)


@pytest.mark.parametrize("D", [128, 512])
def test_rows_without_keys_and_empty_sequences(w4, D):
    got, _ = check(w4, 40, [3, 0, 5, 2], [0, 7, 2, 0], 4, 2, D)
    assert not got[:3].any() and not got[3:6].any() and not got[8:10].any()
    assert got[6:8].any()


def test_many_short_sequences(w4):
    rng = np.random.default_rng(5)
    lq = rng.integers(0, 6, 300)
    lq[100:140] = 0
    check(w4, 50, lq.tolist(), (lq + rng.integers(0, 140, 300)).tolist(), 2, 1, 128)


@pytest.mark.parametrize("D", [128, 256])
def test_sharp_and_growing_scores(w4, D):
    """Large scales (one key takes all) and scores that grow along the keys, so that
    the reference maximum moves many times."""
    import torch
    check(w4, 60, [90], [90], 4, 1, D, scale=1.0)
    q, k, v, cu_q, cu_k = make(61, [64], [900], 4, 1, D)
    k = (k.float() * torch.linspace(0.01, 3.0, 900)[:, None, None]).bfloat16()
    got = run(w4, q, k, v, cu_q, cu_k, 0, 0.5)
    qf, kf, vf = (x.float().numpy().astype(np.float64) for x in (q, k, v))
    ref, ab = draft.attn_prompt(qf, kf, vf, cu_q, cu_k, 0, 0.5)
    S = 0.5 * float(np.sqrt((qf ** 2).sum(-1).max() * (kf ** 2).sum(-1).max()))
    assert (np.abs(got - ref) <= rel_bound(D, S, 900) * ab + 1e-30).all()


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_nothing_leaks_between_rows(w4, D):
    """NaN and infinities in other sequences, in later tokens and before the window:
    rows that do not keep them are bitwise as without, rows that do are not finite."""
    import torch
    lq, lk, window = [50, 60], [50, 250], 90
    q, k, v, cu_q, cu_k = make(70, lq, lk, 8, 2, D)
    clean = run(w4, q, k, v, cu_q, cu_k, window, D ** -0.5)
    bad_k = {50 + 210: float("nan"), 20: float("inf"), 50 + 105: float("nan")}
    for where, val in bad_k.items():
        for x in ("k", "v"):
            k2, v2 = k.clone(), v.clone()
            (k2 if x == "k" else v2)[where] = val
            got = run(w4, q, k2, v2, cu_q, cu_k, window, D ** -0.5)
            for b in range(2):
                for i in range(lq[b]):
                    p = lk[b] - lq[b] + i
                    t = where - cu_k[b]
                    kept = 0 <= t < lk[b] and p - window < t <= p
                    row = cu_q[b] + i
                    if not kept:
                        np.testing.assert_array_equal(got[row], clean[row], err_msg=f"{x}[{where}] row {row}")
                    elif x == "v" or np.isnan(val):
                        assert not np.isfinite(got[row]).any(), f"{x}[{where}] row {row}"
    # one column of one value row only
    v2 = v.clone()
    v2[50 + 220, 1, 3] = float("-inf")
    got = run(w4, q, k, v2, cu_q, cu_k, window, D ** -0.5)
    for i in range(60):
        kept = 190 + i >= 220
        row = got[50 + i]
        if kept:
            assert np.all(row[4:, 3] == -np.inf)
            row, want = np.delete(row, 3, 1), np.delete(clean[50 + i], 3, 1)
        else:
            want = clean[50 + i]
        np.testing.assert_array_equal(row, want)


def test_strided_views(w4):
    """q, k and v as views of one fused projection, out inside a wider buffer."""
    import torch
    T, Hq, Hkv, D = 150, 8, 2, 128
    g = torch.Generator().manual_seed(8)
    wide = torch.randn(T, (Hq + 2 * Hkv) * D + 8, generator=g).bfloat16().cuda()
    q = wide[:, :Hq * D].view(T, Hq, D)
    k = wide[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = wide[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(T, Hkv, D)
    cu = torch.tensor([0, 100, T], dtype=torch.int32, device="cuda")
    want = w4.w4_attn_prompt(q.contiguous(), k.contiguous(), v.contiguous(), cu, scale=0.1)
    ob = torch.full((T, Hq * D + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got = w4.w4_attn_prompt(q, k, v, cu, scale=0.1, out=ob[:, :Hq * D].view(T, Hq, D))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool((ob[:, Hq * D:] == 7.0).all())


def test_rows_of_no_sequence_are_not_written(w4):
    import torch
    q, k, v, cu_q, cu_k = make(80, [30, 30, 30], [30, 30, 30], 4, 1, 128)
    g = Guard((90, 4, 128), torch.bfloat16)
    g.t.fill_(5.0)
    # the second sequence alone, and lengths that pass the end are cut there
    for cu in ([30, 60], [60, 200]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        w4.w4_attn_prompt(q.cuda(), k.cuda(), v.cuda(), c, out=g.t)
        torch.cuda.synchronize()
        g.check("part")
    got = g.t.float().cpu().numpy()
    assert (got[:30] == 5.0).all() and np.isfinite(got).all() and not (got[30:] == 5.0).all(-1).any()


def test_deterministic_streams_and_graphs(w4):
    """The same bits again, on another stream, and from a captured call whose
    lengths change on the device."""
    import torch
    lens = [[200, 313, 7], [1, 500, 19]]
    q, k, v, cu_a, _ = make(90, lens[0], lens[0], 8, 2, 256)
    cu_b = np.concatenate([[0], np.cumsum(lens[1])]).astype(np.int32)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    want = [torch.from_numpy(run(w4, q, k, v, c, None, 0, 0.1)) for c in (cu_a, cu_b)]
    cu = torch.from_numpy(cu_a).cuda()
    out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w4.w4_attn_prompt(q, k, v, cu, scale=0.1, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out.double().cpu(), want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4_attn_prompt(q, k, v, cu, scale=0.1, out=out, stream=s)
    for c, w in ((cu_b, want[1]), (cu_a, want[0])):
        out.zero_()
        cu.copy_(torch.from_numpy(c))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.double().cpu(), w)
    assert w4.device_error() == 0


def test_binding_checks(w4):
    import torch
    q = torch.zeros(4, 8, 256, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(4, 1, 256, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for bad in (lambda: w4.w4_attn_prompt(q.float(), kv, kv, cu), lambda: w4.w4_attn_prompt(q, kv, kv[:3], cu),
                lambda: w4.w4_attn_prompt(q, kv, kv, cu.long()), lambda: w4.w4_attn_prompt(q, kv, kv, cu, cu[:1]),
                lambda: w4.w4_attn_prompt(q.transpose(0, 1), kv, kv, cu),
                lambda: w4.w4_attn_prompt(q, kv, kv, cu, out=q[:3])):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(w4.W4Error):
        w4.w4_attn_prompt(q, kv, kv, cu, scale=0.0)
    with pytest.raises(w4.W4Error):
        w4.w4_attn_prompt(q[:, :, :96].contiguous(), kv[:, :, :96].contiguous(), kv[:, :, :96].contiguous(), cu)

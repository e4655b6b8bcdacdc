"""Log probabilities, entropy and alternatives against the fp64 statement.

Bounds: a logit minus the row's maximum and the logarithm of the sum are fp32
(2^-23 relative each), exp2 of the hardware is within 2^-22 and its argument's
rounding within 2^-23 |x - m| log2 e, all of which move the sum of probabilities by
at most 2^-20 for |x - m| <= 40 where it counts, and fp32 sums of V terms in blocks
of 64 add log2(V) 2^-24 or so: 2^-18 absolute on log s and on the entropy's two
parts, plus 2^-22 of each value. Indices are exact.
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


def run(w4, x, targets, topk, status=False):
    import torch
    M, V = x.shape
    x = x if x.is_cuda else x.cuda()
    gs = [Guard((M,), torch.float32), Guard((M,), torch.float32), Guard((M, topk), torch.float32) if topk else None,
          Guard((M, topk), torch.int32) if topk else None]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = None if targets is None else torch.from_numpy(np.asarray(targets, np.int32)).cuda()
    out = [g.t if g is not None else None for g in gs]
    if t is None:
        out[0] = None
    w4.w4_logprobs(x, t, topk, status=st if status else None, out=out)
    torch.cuda.synchronize()
    for g in gs:
        if g is not None:
            g.check("w4_logprobs")
    r = [None if o is None else o.cpu().numpy() for o in out]
    return r + [int(st.item())]


def check(w4, x, targets, topk):
    lp, ent, top, ids, st = run(w4, x, targets, topk, True)
    rl, re, rt, ri, rs = draft.logprobs(x.float().cpu().numpy(), targets, topk)
    assert st == rs

    def near(a, b):
        a = a.astype(np.float64)
        fin = np.isfinite(b)
        np.testing.assert_array_equal(a[~fin], b[~fin])
        assert (np.abs(a[fin] - b[fin]) <= 2.0 ** -18 + 2.0 ** -22 * np.abs(b[fin])).all()

    near(ent, re)
    if targets is not None:
        near(lp, rl)
    if topk:
        np.testing.assert_array_equal(ids, ri)
        near(top, rt)
    return lp, ent, top, ids


def logits(seed, M, V, scale=3.0):
    import torch
    return torch.randn(M, V, generator=torch.Generator().manual_seed(seed)) * scale


@pytest.mark.parametrize("M,V,k", [(1, 1, 1), (2, 3, 5), (1, 255, 32), (3, 256, 20), (2, 257, 1), (5, 1000, 0),
                                   (7, 32003, 20), (1, 262144, 32), (16, 50001, 5)])
def test_sizes(w4, M, V, k):
    rng = np.random.default_rng(V)
    check(w4, logits(V, M, V), rng.integers(0, V, M), k)


@pytest.mark.parametrize("M,V,k", [(1, 262145, 32), (2, 300007, 7), (1, 700001, 32), (1, 2000003, 3)])
def test_rows_of_many_chunks(w4, M, V, k):
    """More chunk maxima than the finishing block's threads hold at once, and more
    blocks' worth of chunks than it has threads."""
    x = logits(V, M, V)
    check(w4, x, [V - 1] * M, k)
    x[0] = float("-inf")
    x[0, ::4096] = 1.0            # the last chunks' too: equal logits, one per 16 chunks
    x[-1, V - 1] = 50.0
    check(w4, x, [V - 1] * M, k)


@pytest.mark.parametrize("k", [1, 5, 32])
def test_best_chunks_in_one_thread(w4, k):
    """The best logits 256 chunks apart: one thread's share holds all of them."""
    x = logits(12, 1, 600000)
    x[0, 77:600000:65536] += 100.0
    check(w4, x, [77], k)
    x[0, 1024:1024 + 256 * 3] = 90.0   # three chunks of equal logits
    check(w4, x, [77], k)


def test_strided_rows_of_every_alignment(w4):
    import torch
    for off in range(4):
        wide = logits(off, 5, 3000).cuda()
        x = wide[:, off:off + 2501]
        check(w4, x, [0, 2500, 1, 7, 1250], 9)


def test_ties_and_signed_zeros(w4):
    import torch
    x = torch.zeros(3, 5000)
    x[0, 1::2] = -0.0
    x[1] = 2.5
    x[2, 4000:] = 1.0
    x[2, 300] = 1.0
    _, ent, _, ids = check(w4, x, [4, 4999, 300], 32)
    assert ids[0].tolist() == list(range(32)) and ids[2].tolist() == [300] + list(range(4000, 4031))
    assert abs(ent[1] - np.log(5000)) < 1e-5


def test_few_allowed_tokens(w4):
    """A constrained decoder's mask: fewer finite logits than alternatives asked for."""
    import torch
    x = torch.full((3, 70000), float("-inf"))
    x[0, [5, 69999, 31000]] = torch.tensor([1.0, 3.0, 3.0])
    x[1, 123] = -200.0
    lp, ent, top, ids = check(w4, x, [5, 7, 0], 8)
    assert ids[0][:4].tolist() == [31000, 69999, 5, 0] and lp[1] == -np.inf and ent[1] == 0 and ent[2] == 0
    assert ids[2].tolist() == list(range(8)) and np.all(top[2] == -np.inf)


def test_nan_and_infinity(w4):
    import torch
    x = logits(3, 4, 9000)
    x[0, 8999] = float("nan")
    x[1, 0] = float("inf")
    x[2] = float("nan")
    lp, ent, top, ids = check(w4, x, [1, 1, 1, 1], 4)
    assert np.isnan(lp[:3]).all() and np.isnan(ent[:3]).all() and (ids[:3] == -1).all() and np.isfinite(lp[3])


def test_wide_and_extreme_logits(w4):
    import torch
    x = logits(4, 3, 40000, 40.0)
    x[1] -= 1e6
    x[2] = torch.linspace(-3e38, 3e38, 40000, dtype=torch.float64).float()  # the step overflows fp32
    lp, ent, top, ids = run(w4, x, [10, 20, 39999], 5)[:4]
    rl, re, rt, ri, _ = draft.logprobs(x.numpy(), [10, 20, 39999], 5)
    np.testing.assert_array_equal(ids, ri)
    assert np.abs(ent - re).max() < 1e-3 and np.abs(lp[:2] - rl[:2]).max() < 0.2 and lp[2] == 0


def test_ascending_and_descending(w4):
    import torch
    x = torch.stack([torch.arange(100000.0), -torch.arange(100000.0)]) / 1000
    check(w4, x, [0, 0], 32)


def test_targets_out_of_range(w4):
    lp, _, _, _, st = run(w4, logits(5, 4, 1000), [-1, 1000, 3, 2 ** 31 - 1], 0, True)
    assert st == 1 and lp[0] == lp[1] == lp[3] == 0 and lp[2] < 0
    assert run(w4, logits(5, 4, 1000), [0, 999, 3, 4], 0, True)[4] == 0


def test_more_rows_than_one_pass(w4):
    M, V = 70000, 40
    x = logits(6, M, V)
    check(w4, x, np.arange(M) % V, 2)


def test_optional_outputs(w4):
    import torch
    x = logits(7, 3, 5000).cuda()
    full = w4.w4_logprobs(x, torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda"), 6)
    lp, ent, top, ids = w4.w4_logprobs(x, topk=6)
    assert lp is None and torch.equal(ids, full[3]) and torch.equal(top, full[2]) and torch.equal(ent, full[1])
    only = torch.empty((3, 6), dtype=torch.int32, device="cuda")
    w4.w4_logprobs(x, topk=6, out=(None, None, None, only))
    assert torch.equal(only, full[3])


def test_graph_and_determinism(w4):
    import torch
    x = logits(8, 8, 262144).cuda()
    t = torch.arange(8, dtype=torch.int32, device="cuda")
    a = w4.w4_logprobs(x, t, 20)
    out = [torch.zeros_like(y) for y in a]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4_logprobs(x, t, 20, out=out, stream=s)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, out))


def test_refusals(w4):
    import torch
    x = logits(9, 2, 100).cuda()
    for bad in (lambda: w4.w4_logprobs(x.half()), lambda: w4.w4_logprobs(x.t()), lambda: w4.w4_logprobs(x[0]),
                lambda: w4.w4_logprobs(x, torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: w4.w4_logprobs(x, torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for k in (33, -1):
        with pytest.raises(w4.W4Error):
            w4.w4_logprobs(x, topk=k)


def test_captured_calls_between_newer_ones(w4):
    """A captured call is replayed after many newer calls on the same rows, and they
    after it."""
    import torch
    x = logits(20, 5, 60000).cuda()
    t = torch.arange(5, dtype=torch.int32, device="cuda")
    want = w4.w4_logprobs(x, t, 7)
    out = [torch.zeros_like(y) for y in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4_logprobs(x, t, 7, out=out, stream=s)
    for n in (1, 3, 2000):  # blocks per row differ with the rows' number and length
        other = logits(n, n, 300).cuda()
        for _ in range(4):
            w4.w4_logprobs(other, topk=3)
            [y.zero_() for y in out]
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
            got = w4.w4_logprobs(x, t, 7)
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_that_overlapped_leave_nothing_behind(w4):
    """Calls that break the rule and overlap on two streams may give anything (inside
    their outputs); a call after them is right, and after it a captured one."""
    import torch
    xs = [logits(21, 4, 262144).cuda(), logits(22, 3, 70001).cuda(), logits(23, 40, 9000).cuda()]
    want = [w4.w4_logprobs(x, topk=5) for x in xs]
    outs = [[(Guard((x.shape[0],), torch.float32), Guard((x.shape[0], 5), torch.float32),
              Guard((x.shape[0], 5), torch.int32)) for x in xs] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    s = torch.cuda.Stream()
    cap = [torch.zeros_like(y) for y in want[0][1:]]
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w4.w4_logprobs(xs[0], topk=5, out=(None, *cap), stream=s)
    torch.cuda.synchronize()
    for turn in range(30):
        for i in range(6):
            for j in range(2):
                n = (i + j + turn) % 3
                w4.w4_logprobs(xs[n], topk=5, out=(None, *(b.t for b in outs[j][n])), stream=streams[j])
        torch.cuda.synchronize()
        for o in outs:
            for gs in o:
                for b in gs:
                    b.check("overlapping calls")
        for x, w in zip(xs, want):
            got = w4.w4_logprobs(x, topk=5)
            assert all(torch.equal(a, b) for a, b in zip(got[1:], w[1:]))
    for i in range(6):
        for j in range(2):
            w4.w4_logprobs(xs[(i + j) % 3], topk=5, out=(None, *(b.t for b in outs[j][(i + j) % 3])), stream=streams[j])
    torch.cuda.synchronize()
    big = logits(24, 40, 500).cuda()  # rows of every call above
    assert torch.equal(w4.w4_logprobs(big, topk=1)[3][:, 0].long(), big.argmax(1))
    assert w4.device_error() == 0
    [y.zero_() for y in cap]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(cap, want[0][1:]))

"""Long caches, whose one row tile is cut over all SMs and merged from that many parts.

Exact form: queries of zeros weigh every kept key alike (each weight is exactly 1), and
values of 0 and +-1 make every sum a small whole number, exact in fp32 in any order. What
is left is a division and the rounding of the output to bf16, 2^-8: a key lost, taken
twice or kept wrongly moves about 1/16 of the columns by one of a sum of about 90.

Random form, by the norm of a row's error: the roundings of the weights are independent
from key to key, so their sum grows as the output does, with the root of the length.
With delta = 2^-8 (weights to bf16) + 2^-15 + 2 D 2^-23 S (scores; both as in the
elementwise bound of the prompt attention), independent and uniform at most, the root mean
square of the error is delta / sqrt(3) sqrt(A), A = sum_t w_t^2 |v_t|^2; twice that is
allowed, then 2^-8 |out| for the output's rounding and 2 (T / 8 + 64) 2^-23 |out| for the
fp32 sums. One lost tile of 128 keys of 130000 is about 0.03 |out|, twice the bound.
"""
import pytest

from test_attn_prompt_parity import w4  # noqa: F401

pytestmark = pytest.mark.gpu


def signs(g, *shape):
    """0 and +-1, one in 16 not zero."""
    import torch
    x = torch.randint(0, 32, shape, generator=g, device="cuda", dtype=torch.int8)
    return ((x == 0).to(torch.bfloat16) - (x == 1).to(torch.bfloat16))


def exact(got, want):
    err = (got.double() - want).abs()
    bound = want.abs() * (2.0 ** -8 + 2.0 ** -20)
    assert bool((err <= bound).all()), f"{int((err > bound).sum())} of {err.numel()} columns off"


def chain_keep(parents):
    """bool [N][N]: ancestors or self of each node."""
    import torch
    N = len(parents)
    keep = torch.zeros(N, N, dtype=torch.bool)
    for i in range(N):
        j = i
        while j >= 0:
            keep[i, j] = True
            j = parents[j]
    return keep.cuda()


@pytest.mark.parametrize("D", [64, 128, 256, 384, 512])
@pytest.mark.parametrize("window", [0, 100003])
def test_tree_keeps_every_key_once(w4, D, window):  # noqa: F811
    import torch
    T, pos, Hkv, G = 131072, 130001, 1, 2
    parents = [-1, 0, 0, 1, 3]
    N = len(parents)
    g = torch.Generator(device="cuda").manual_seed(D)
    q = torch.zeros(1, N, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    k, v = torch.ones(1, T, Hkv, D, dtype=torch.bfloat16, device="cuda"), signs(g, 1, T, Hkv, D)
    kt, vt = torch.ones(1, N, Hkv, D, dtype=torch.bfloat16, device="cuda"), signs(g, 1, N, Hkv, D)
    v[:, pos:] = float("nan")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = w4.w4_attn_tree(q, k, v, kt, vt, i32([parents]), i32([pos]), window=window, scale=0.1)
    keep = chain_keep(parents)
    for i in range(N):
        depth = int(keep[i].sum()) - 1
        lo = pos + depth - window + 1 if window else 0
        s = v[0, lo:pos, 0].double().sum(0) + vt[0, :, 0].double()[keep[i]].sum(0)
        want = s / (pos - lo + depth + 1)
        for h in range(G):
            exact(out[0, i, h], want)
    assert w4.device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256, 384, 512])
def test_ring_keeps_every_key_once(w4, D):  # noqa: F811
    import torch
    T, pos = 65536, 200001
    g = torch.Generator(device="cuda").manual_seed(D + 1)
    q = torch.zeros(1, 3, 2, D, dtype=torch.bfloat16, device="cuda")
    k, v = torch.ones(1, T, 1, D, dtype=torch.bfloat16, device="cuda"), signs(g, 1, T, 1, D)
    kt, vt = torch.ones(1, 3, 1, D, dtype=torch.bfloat16, device="cuda"), signs(g, 1, 3, 1, D)
    slot = torch.arange(T, device="cuda")
    p = pos - 1 - (pos - 1 - slot) % T
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = w4.w4_attn_tree(q, k, v, kt, vt, i32([[-1, 0, 1]]), i32([pos]), kpos=p.int()[None].contiguous(), window=T,
                          scale=0.1)
    for i in range(3):
        kept = p > pos + i - T
        s = v[0, kept, 0].double().sum(0) + vt[0, :i + 1, 0].double().sum(0)
        for h in range(2):
            exact(out[0, i, h], s / (int(kept.sum()) + i + 1))
    assert w4.device_error() == 0


@pytest.mark.parametrize("D", [64, 128, 256, 384, 512])
@pytest.mark.parametrize("lq,window", [(70, 0), (3, 90001)])
def test_chunk_keeps_every_key_once(w4, D, lq, window):  # noqa: F811
    import torch
    lk, G = 130077, 8
    g = torch.Generator(device="cuda").manual_seed(D + 2)
    q = torch.zeros(lq, G, D, dtype=torch.bfloat16, device="cuda")
    k, v = torch.ones(lk, 1, D, dtype=torch.bfloat16, device="cuda"), signs(g, lk, 1, D)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = w4.w4_attn_prompt(q, k, v, i32([0, lq]), i32([0, lk]), window=window, scale=0.1)
    sums = torch.cat([torch.zeros(1, D, dtype=torch.float64, device="cuda"), v[:, 0].double().cumsum(0)])
    at = torch.arange(lk - lq, lk, device="cuda")
    lo = (at - window + 1).clamp(min=0) if window else torch.zeros_like(at)
    want = (sums[at + 1] - sums[lo]) / (at + 1 - lo)[:, None].double()
    exact(out, want[:, None].expand(lq, G, D))
    assert w4.device_error() == 0


def near(got, q, k, v, keep, scale):
    """A row of D query values over kept rows of k and v."""
    import torch
    k, v, q = k[keep].double(), v[keep].double(), q.double()
    T, D = k.shape
    w = torch.softmax(scale * (k @ q), 0)
    out = w @ v
    S = scale * float(q.norm() * k.norm(dim=1).max())
    delta = 2.0 ** -8 + 2.0 ** -15 + 2 * D * 2.0 ** -23 * S
    A = float((w.square() * v.square().sum(1)).sum())
    bound = 2 * delta / 3 ** 0.5 * A ** 0.5 + (2.0 ** -8 + 2 * (T / 8 + 64) * 2.0 ** -23) * float(out.norm())
    err = float((got.double() - out).norm())
    assert err <= bound, f"{err / bound:.3f} of the bound"


@pytest.mark.parametrize("D", [128, 256, 512])
def test_random_values_by_norm(w4, D):  # noqa: F811
    import torch
    T, pos, G = 131072, 130001, 4
    parents = [-1, 0, 1, 0]
    N = len(parents)
    g = torch.Generator(device="cuda").manual_seed(D + 3)
    rnd = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    q, k, v, kt, vt = rnd(1, N, G, D), rnd(1, T, 1, D), rnd(1, T, 1, D), rnd(1, N, 1, D), rnd(1, N, 1, D)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = w4.w4_attn_tree(q, k, v, kt, vt, i32([parents]), i32([pos]), scale=D ** -0.5)
    allk, allv = torch.cat([k[0, :, 0], kt[0, :, 0]]), torch.cat([v[0, :, 0], vt[0, :, 0]])
    chains = chain_keep(parents)
    for i in range(N):
        keep = torch.cat([torch.arange(T, device="cuda") < pos, chains[i]])
        for h in range(G):
            near(out[0, i, h], q[0, i, h], allk, allv, keep, D ** -0.5)
    lq, lk = 33, 130033
    qc = rnd(lq, G, D)
    out = w4.w4_attn_prompt(qc, k[0, :lk], v[0, :lk], i32([0, lq]), i32([0, lk]), scale=D ** -0.5)
    for i in (0, 15, 16, 31, 32):
        keep = torch.arange(lk, device="cuda") <= lk - lq + i
        for h in range(G):
            near(out[i, h], qc[i, h], k[0, :lk, 0], v[0, :lk, 0], keep, D ** -0.5)
    assert w4.device_error() == 0

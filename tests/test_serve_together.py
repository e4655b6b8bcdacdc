"""Several requests through one layer: projections with adapters, norms with rotation into
a paged cache, attention; prompts in chunks first, then single tokens from a captured
graph whose lengths and tables live on the device. Every stage is compared with the fp64
statement of it on what the stage before left (bounds as in the stages' own tests)."""
import numpy as np
import pytest

import synth
from oracle import serve

pytestmark = pytest.mark.gpu

K, HQ, HKV, D, PAGE, WINDOW, R, L = 512, 8, 2, 128, 16, 90, 16, 3
N = (HQ + 2 * HKV) * D


@pytest.fixture(scope="module")
def w4():
    import bit_weight_only_w4a16_gb300 as w4
    w4.init()
    return w4


def dev(a, dt=np.int32):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()


def f64(t):
    return t.double().cpu().numpy()


class Layer:
    def __init__(self, seed):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*s):
            return torch.randn(*s, generator=g, device="cuda")
        _, qw, sc = synth.gen_w4_problem(seed, 1, N, K)
        self.qw, self.sc = dev(qw.view(np.int32)), dev(sc.view(np.int16), np.int16)
        self.a, self.b = (randn(L, R, K) * K ** -0.5).bfloat16(), (randn(L, N, R) * 0.3).bfloat16()
        self.s = 0.5 + torch.rand(L, generator=g, device="cuda")
        self.nq, self.nk = 1 + 0.2 * randn(D), 1 + 0.2 * randn(D)
        self.f = dev(1e4 ** (-np.arange(0, D, 2) / D), np.float32)
        self.kp = randn(40, PAGE, HKV, D).bfloat16()
        self.vp = randn(40, PAGE, HKV, D).bfloat16()

    def run(self, w4, x, ids, table, lens, cu=None, stream=None):
        M = x.shape[0]
        y = w4.w4a16_gemm(x, self.qw, self.sc, stream=stream)
        z = w4.w4_lora(y, x, self.a, self.b, ids, scale=self.s, stream=stream)
        q, k, v = (z[:, i * D:j * D].view(M, j - i, D) for i, j in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
        qo = w4.w4_qkv_paged(q, k, v, self.kp, self.vp, table, lens, self.f, cu_q=cu, q_weight=self.nq, k_weight=self.nk,
                             stream=stream)
        o = w4.w4_attn_paged(qo, self.kp, self.vp, table, lens, cu_q=cu, window=WINDOW, scale=D ** -0.5, stream=stream)
        return y, z, qo, o

    def check(self, x, ids, table, lens, cu, before, got):
        y, z, qo, o = got
        M = x.shape[0]
        ids, table, lens = (t.cpu().numpy() for t in (ids, table, lens))
        cu = None if cu is None else cu.cpu().numpy()
        ref, size, low, _ = serve.lora(f64(y), f64(x), f64(self.a), f64(self.b), ids, f64(self.s))
        assert (np.abs(f64(z) - ref) <= 2.0 ** -16 * low + (K + 2 * R + 40) * 2.0 ** -24 * size).all()
        heads = f64(z).reshape(M, HQ + 2 * HKV, D)
        seq, pos = serve.rows_of(cu, lens, M)
        assert (seq >= 0).all()
        kp, vp = f64(self.kp), f64(self.vp)
        want_k, want_v = before
        for part, w, name in ((slice(0, HQ), self.nq, "q"), (slice(HQ, HQ + HKV), self.nk, "k")):
            t, size = serve.turn(serve.norm(heads[:, part], f64(w), 1e-6), pos, self.f.cpu().numpy(), False)
            bound = 2.0 ** -8 * np.abs(t) + 2.0 ** -19 * (1 + 2.0 ** -8) * size
            at = [serve.place(table, kp.shape[0], PAGE, s, p) for s, p in zip(seq, pos)]
            have = f64(qo) if name == "q" else np.stack([kp[a] for a in at])
            assert (np.abs(have - t) <= bound).all()
        left = np.ones(kp.shape[:2], bool)
        for m, a in enumerate(at):
            left[a] = False
            np.testing.assert_array_equal(vp[a], f64(z[m, (HQ + HKV) * D:].bfloat16()).reshape(HKV, D))
        np.testing.assert_array_equal(kp[left], want_k[left])
        np.testing.assert_array_equal(vp[left], want_v[left])
        ref, ab = serve.attn_paged(f64(qo), kp, vp, table, lens, cu, WINDOW, D ** -0.5)
        S = D ** -0.5 * float(np.sqrt((f64(qo) ** 2).sum(-1).max() * (kp ** 2).sum(-1).max()))
        rel = 2.0 ** -7 + 2.0 ** -15 + 2 * D * 2.0 ** -23 * S + (lens.max() / 8 + 64) * 2.0 ** -23
        assert (np.abs(f64(o) - ref) <= rel * ab + 1e-30).all()


def test_chunks_then_tokens(w4):
    import torch
    layer = Layer(3)
    g = torch.Generator(device="cuda").manual_seed(5)

    def x_of(M):
        return torch.randn(M, K, generator=g, device="cuda").bfloat16()
    order = np.random.default_rng(1).permutation(40).reshape(4, 10)
    table = dev(order)                  # room for 160 positions of each of four requests
    done = np.zeros(4, int)
    owner = np.array([2, -1, 0, 1])     # the requests' adapters
    for lq in ([70, 3, 0, 40], [1, 60, 33, 64]):
        done = done + lq
        cu, lens = dev(np.concatenate([[0], np.cumsum(lq)])), dev(done)
        x, ids = x_of(sum(lq)), dev(np.repeat(owner, lq))
        before = f64(layer.kp), f64(layer.vp)
        got = layer.run(w4, x, ids, table, lens, cu)
        layer.check(x, ids, table, lens, cu, before, got)
    # one captured step serves every token
    x, ids, lens = x_of(4), dev(owner), dev(done)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        with torch.cuda.stream(s):
            lens += 1
            out = layer.run(w4, x, ids, table, lens, stream=s)
    for _ in range(12):
        x.copy_(x_of(4))
        torch.cuda.synchronize()
        before = f64(layer.kp), f64(layer.vp)
        graph.replay()
        torch.cuda.synchronize()
        done = done + 1
        assert lens.tolist() == done.tolist()
        layer.check(x, ids, table, lens, None, before, out)
    assert w4.device_error() == 0


def test_a_request_alone_and_in_a_batch(w4):
    """What other requests hold does not reach a request: its rows are the same bits when theirs change."""
    import torch
    a, b = Layer(4), Layer(4)
    g = torch.Generator(device="cuda").manual_seed(6)
    table, lens = dev(np.arange(40).reshape(4, 10)), dev([30, 5, 150, 1])
    x, ids = torch.randn(4, K, generator=g, device="cuda").bfloat16(), dev([1, 1, 0, -1])
    first = a.run(w4, x, ids, table, lens)
    x2 = x.clone()
    x2[2] = 0
    b.kp[20:30] = float("nan")
    b.vp[20:30] = float("inf")
    second = b.run(w4, x2, ids, table, lens)
    for u, v in zip(first, second):
        for m in (0, 1, 3):
            assert torch.equal(u[m], v[m])
    assert not torch.isfinite(second[3][2]).all()

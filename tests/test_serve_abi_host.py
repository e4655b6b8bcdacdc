"""Refusals of the serving calls: bad arguments are answered on the host, before any
device is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    import bit_weight_only_w4a16_gb300 as w4
    return w4._lib


A = ctypes.c_void_p(1 << 20)  # a plausible, aligned device address; never dereferenced on refusal
O8 = ctypes.c_void_p((1 << 20) + 8)
O2 = ctypes.c_void_p((1 << 20) + 2)
F = ctypes.c_float


def _rope(lib, qo=A, ko=A, q=A, k=A, qw=A, kw=A, f=A, pos=A, M=4, Hq=8, Hkv=1, D=256, R=256, ldq=2048, ldk=256, ldqo=2048,
          ldko=256, f32=1, pairs=0, eps=1e-6):
    return lib.w4_qk_norm_rope(qo, ko, q, k, qw, kw, f, pos, M, Hq, Hkv, D, R, ldq, ldk, ldqo, ldko, f32, pairs, F(eps),
                               None)


@pytest.mark.parametrize("kw,rc", [
    (dict(qo=None), 1), (dict(ko=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(f=None), 1), (dict(pos=None), 1),
    (dict(M=0), 1), (dict(Hq=0), 1), (dict(Hkv=-1), 1), (dict(R=-8), 1), (dict(R=264), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(ldq=2040), 1), (dict(ldk=248), 1),
    (dict(ldqo=1 << 31), 1), (dict(ldko=0), 1), (dict(Hq=1 << 20, ldq=1 << 28, ldqo=1 << 28), 1),
    (dict(D=96), 2), (dict(D=1024, ldq=8192, ldqo=8192, ldk=1024, ldko=1024), 2), (dict(R=100), 2), (dict(R=4), 2),
    (dict(q=O8), 3), (dict(k=O8), 3), (dict(qo=O8), 3), (dict(ko=O8), 3), (dict(qw=O8), 3), (dict(kw=O8), 3),
    (dict(f=O2), 3), (dict(pos=O2), 3), (dict(ldq=2052), 3), (dict(ldko=260), 3),
])
def test_rope_refusals(lib, kw, rc):
    assert _rope(lib, **kw) == rc


def _qkv(lib, qo=A, kp=A, vp=A, q=A, k=A, v=A, qw=A, kw=A, vw=A, f=A, table=A, lens=A, cu=A, B=2, M=4, Hq=8, Hkv=1, D=256,
         R=256, pages=9, page=16, tp=4, ldq=2048, ldk=256, ldv=256, ldqo=2048, ps=4096, rs=256, hs=256, f32=1, pairs=0,
         eps=1e-6, status=None):
    return lib.w4_qkv_paged(qo, kp, vp, q, k, v, qw, kw, vw, f, table, lens, cu, B, M, Hq, Hkv, D, R, pages, page, tp, ldq,
                            ldk, ldv, ldqo, ps, rs, hs, f32, pairs, F(eps), status, None)


PAGES = [
    (dict(pages=0), 1), (dict(page=0), 1), (dict(tp=0), 1), (dict(B=0), 1), (dict(B=4097), 2), (dict(page=8), 2),
    (dict(page=24), 2), (dict(page=2048), 2), (dict(tp=1 << 27), 2), (dict(page=1024, tp=(1 << 21) - 1, rs=256, ps=1 << 18), 2),
    (dict(hs=248), 1), (dict(rs=8), 1), (dict(ps=1024), 1), (dict(ps=256, rs=512), 1), (dict(ps=1 << 39), 1),
    (dict(rs=260, ps=8192), 3), (dict(ps=4100), 3),
]


@pytest.mark.parametrize("kw,rc", PAGES + [
    (dict(qo=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(f=None), 1), (dict(Hkv=0), 1), (dict(cu=None), 1), (dict(M=0), 1),
    (dict(ldv=248), 1), (dict(D=80), 2),
    (dict(v=O8), 3), (dict(kp=O8), 3), (dict(vp=O8), 3), (dict(vw=O8), 3), (dict(table=O2), 3), (dict(lens=O2), 3),
    (dict(cu=O2), 3), (dict(status=O2), 3), (dict(ldv=260), 3),
])
def test_qkv_refusals(lib, kw, rc):
    assert _qkv(lib, **kw) == rc


def _attn(lib, out=A, q=A, kp=A, vp=A, table=A, lens=A, cu=A, B=2, M=4, Hq=8, Hkv=1, D=256, pages=9, page=16, tp=4, ldq=2048,
          ldo=2048, ps=4096, rs=256, hs=256, window=0, scale=1.0):
    return lib.w4_attn_paged(out, q, kp, vp, table, lens, cu, B, M, Hq, Hkv, D, pages, page, tp, ldq, ldo, ps, rs, hs,
                             window, F(scale), None)


@pytest.mark.parametrize("kw,rc", PAGES + [
    (dict(out=None), 1), (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(table=None), 1),
    (dict(lens=None), 1), (dict(cu=None), 1), (dict(M=0), 1), (dict(Hq=0), 1), (dict(Hkv=3), 1), (dict(window=-1), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(ldq=2040), 1), (dict(ldo=1 << 31), 1),
    (dict(D=96), 2), (dict(Hq=129, ldq=129 * 256, ldo=129 * 256), 2), (dict(M=2**31 - 1024), 2),
    (dict(q=O8), 3), (dict(out=O8), 3), (dict(kp=O8), 3), (dict(vp=O8), 3), (dict(table=O2), 3), (dict(lens=O2), 3),
    (dict(cu=O2), 3), (dict(ldq=2052), 3),
])
def test_attn_refusals(lib, kw, rc):
    assert _attn(lib, **kw) == rc


def _lora(lib, out=A, y=A, x=A, a=A, b=A, ids=A, scale=A, M=3, N=64, K=96, R=16, L=2, ldo=64, ldy=64, ldx=96, status=None):
    return lib.w4_lora(out, y, x, a, b, ids, scale, M, N, K, R, L, ldo, ldy, ldx, status, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(out=None), 1), (dict(y=None), 1), (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(ids=None), 1),
    (dict(M=0), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(R=0), 1), (dict(L=0), 1), (dict(N=60), 1), (dict(K=80), 1),
    (dict(ldo=60), 1), (dict(ldy=60), 1), (dict(ldx=88), 1), (dict(ldo=68), 1), (dict(ldy=1 << 31), 1),
    (dict(R=12), 2), (dict(R=136), 2), (dict(N=(1 << 23) + 8, ldo=1 << 24, ldy=1 << 24), 2),
    (dict(out=O8), 3), (dict(y=O8), 3), (dict(x=O8), 3), (dict(a=O8), 3), (dict(b=O8), 3), (dict(ids=O2), 3),
    (dict(scale=O2), 3), (dict(status=O2), 3), (dict(ldo=66, ldy=66), 3), (dict(ldx=100), 3),
])
def test_lora_refusals(lib, kw, rc):
    assert _lora(lib, **kw) == rc


def test_orders_of_strides(lib):
    """Heads before rows, and keys and values of a page side by side, are served."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (_qkv, _attn):
        kw = dict(Hq=8, Hkv=2, D=128, ldq=1024, ldk=256, ldv=256, ldqo=1024) if call is _qkv else \
            dict(Hq=8, Hkv=2, D=128, ldq=1024, ldo=1024)
        kw.update({} if call is _attn else dict(R=128))
        assert call(lib, **kw, ps=16 * 256, rs=256, hs=128) == 5
        assert call(lib, **kw, ps=16 * 256, rs=128, hs=16 * 128) == 5
        assert call(lib, **kw, ps=2 * 16 * 256, rs=256, hs=128) == 5
        assert call(lib, **kw, ps=256, rs=9 * 256, hs=128) == 5            # pages innermost
        assert call(lib, **kw, ps=16 * 256, rs=128, hs=15 * 128) == 1      # heads overlap
        assert call(lib, **kw, ps=16 * 256 - 8, rs=256, hs=128) == 1       # pages overlap


def test_no_device_after_the_checks(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _rope(lib) == 5 and _rope(lib, qw=None, kw=None) == 5 and _rope(lib, R=0, f=None) == 5
    assert _rope(lib, Hkv=0, k=None, ko=None, ldk=0, ldko=0) == 5
    assert _qkv(lib) == 5 and _qkv(lib, cu=None, M=2) == 5 and _qkv(lib, status=A, vw=None) == 5
    assert _lora(lib) == 5 and _lora(lib, scale=None, status=A) == 5 and _lora(lib, M=2**31 - 1, N=1 << 23, ldo=1 << 23,
                                                                               ldy=1 << 23, R=128) == 5
    assert _attn(lib) == 5 and _attn(lib, cu=None, M=2) == 5
    assert _attn(lib, page=1024, tp=(1 << 21) - 2, ps=1 << 18) == 5


def test_binding_refuses_host_tensors():
    import torch
    import bit_weight_only_w4a16_gb300 as w4
    q, kv = torch.zeros(2, 8, 256), torch.zeros(2, 1, 256)
    pages = torch.zeros(3, 16, 1, 256, dtype=torch.bfloat16)
    t, i = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    f = torch.ones(128)
    with pytest.raises(ValueError):
        w4.w4_qk_norm_rope(q, kv, i, f)
    with pytest.raises(ValueError):
        w4.w4_qkv_paged(q, kv, kv, pages, pages, t, i, f)
    with pytest.raises(ValueError):
        w4.w4_lora(torch.zeros(2, 8), q[:, 0].bfloat16(), pages[:2, :8, 0], pages[:2, :8, 0, :8], i)
    with pytest.raises(ValueError):
        w4.w4_attn_paged(q.bfloat16(), pages, pages, t, i)

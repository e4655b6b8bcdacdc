"""Refusals of the prompt and draft calls: bad arguments are answered on the host,
before any device is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    import bit_weight_only_w4a16_gb300 as w4
    return w4._lib


A = ctypes.c_void_p(1 << 20)  # a plausible, aligned device address; never dereferenced on refusal
O8 = ctypes.c_void_p((1 << 20) + 8)
O2 = ctypes.c_void_p((1 << 20) + 2)


def _prompt(lib, out=A, q=A, k=A, v=A, cu_q=A, cu_k=A, B=1, Sq=16, Sk=16, Hq=8, Hkv=1, D=256, ldq=2048, ldk=256,
            ldv=256, ldo=2048, window=0, scale=1.0):
    return lib.w4_attn_prompt(out, q, k, v, cu_q, cu_k, B, Sq, Sk, Hq, Hkv, D, ldq, ldk, ldv, ldo, window,
                              ctypes.c_float(scale), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(out=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(cu_q=None), 1),
    (dict(B=0), 1), (dict(Sq=0), 1), (dict(Sk=0), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hkv=3), 1),
    (dict(window=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(ldq=2040), 1), (dict(ldk=248), 1), (dict(ldo=1 << 31), 1),
    (dict(B=4097), 2), (dict(D=96), 2), (dict(D=192), 2), (dict(D=1024, ldq=8192, ldk=1024, ldv=1024, ldo=8192), 2),
    (dict(Hq=129, ldq=129 * 256, ldo=129 * 256), 2),
    (dict(q=O8), 3), (dict(k=O8), 3), (dict(v=O8), 3), (dict(out=O8), 3), (dict(cu_q=O2), 3), (dict(cu_k=O2), 3),
    (dict(ldq=2052), 3), (dict(ldv=260), 3),
])
def test_prompt_refusals(lib, kw, rc):
    assert _prompt(lib, **kw) == rc


def _tree(lib, out=A, q=A, k=A, v=A, kpos=None, kt=A, vt=A, parents=A, pos=A, B=1, N=8, T=512, Hq=8, Hkv=1, D=256,
          window=0, scale=1.0):
    return lib.w4_attn_tree(out, q, k, v, kpos, kt, vt, parents, pos, B, N, T, Hq, Hkv, D, window,
                            ctypes.c_float(scale), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(out=None), 1), (dict(kt=None), 1), (dict(vt=None), 1), (dict(parents=None), 1), (dict(pos=None), 1),
    (dict(N=0), 1), (dict(T=0), 1), (dict(B=0), 1), (dict(B=4096, T=1 << 20), 1), (dict(scale=0.0), 1),
    (dict(window=-5), 1), (dict(Hq=6, Hkv=4), 1),
    (dict(N=65), 2), (dict(B=5000), 2), (dict(D=80), 2), (dict(Hq=256), 2),
    (dict(kt=O8), 3), (dict(kpos=O2), 3), (dict(parents=O2), 3), (dict(pos=O2), 3),
])
def test_tree_refusals(lib, kw, rc):
    assert _tree(lib, **kw) == rc


def _logprobs(lib, lp=A, ent=A, top=A, ids=A, x=A, t=A, M=1, V=100, ld=100, k=5, status=None):
    return lib.w4_logprobs(lp, ent, top, ids, x, t, M, V, ld, k, status, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), 1), (dict(t=None), 1), (dict(M=0), 1), (dict(V=0), 1), (dict(ld=99), 1), (dict(k=-1), 1),
    (dict(lp=None, t=None, ent=None, top=None, ids=None), 1), (dict(lp=None, ent=None, k=0), 1),
    (dict(k=33), 2),
    (dict(x=O2), 3), (dict(t=O2), 3), (dict(top=O2), 3), (dict(status=O2), 3),
])
def test_logprobs_refusals(lib, kw, rc):
    assert _logprobs(lib, **kw) == rc


def test_logprobs_row_of_2_31(lib):
    # chunk numbers and ends are 32-bit: a row must end 1024 before 2^31
    V = 2**31 - 1024
    assert _logprobs(lib, V=V, ld=V) == 2
    assert _logprobs(lib, V=2**31 - 1, ld=2**31 - 1) == 2


@pytest.mark.parametrize("n", [2**31 - 1024, 2**31 - 1])
def test_attention_rows_next_to_2_31(lib, n):
    # a key tile's end is a 32-bit number too
    assert _prompt(lib, Sk=n) == 2 and _prompt(lib, Sq=n) == 2
    assert _tree(lib, T=n) == 2 and _tree(lib, B=2, T=n // 2 + 1) == (2 if n < 2**31 - 1 else 1)


@pytest.mark.parametrize("D,rc", [(64, 5), (256, 5), (512, 2)])
def test_row_tiles_past_2_31(lib, D, rc):
    # 4096 sequences of one token on 2^18 + 1 heads: 2^30 + 4096 row tiles, two slices at D = 512
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    H = (1 << 18) + 1
    assert _prompt(lib, B=4095, Sq=4096, Hq=H, Hkv=H, D=D, ldq=H * D, ldk=H * D, ldv=H * D, ldo=H * D) == rc
    assert _prompt(lib, B=4095, Sq=4096, Hq=2 * H, Hkv=2 * H, D=D, ldq=2 * H * D, ldk=2 * H * D, ldv=2 * H * D,
                   ldo=2 * H * D) == 2
    assert _tree(lib, B=4096, N=1, T=1, Hq=H, Hkv=H, D=D) == rc


def _commit(lib, kc=A, vc=A, kpos=None, kt=A, vt=A, path=A, count=A, pos=A, L=1, B=1, N=8, T=16, W=64, status=None):
    return lib.w4_kv_commit(kc, vc, kpos, kt, vt, path, count, pos, L, B, N, T, W, status, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(kc=None), 1), (dict(vt=None), 1), (dict(path=None), 1), (dict(count=None), 1), (dict(pos=None), 1),
    (dict(L=0), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(T=0), 1), (dict(W=4), 1), (dict(W=100), 1),
    (dict(L=1 << 16, B=1 << 16), 1), (dict(N=65), 2),
    (dict(kt=O8), 3), (dict(kpos=O2), 3), (dict(count=O2), 3), (dict(status=O2), 3),
])
def test_commit_refusals(lib, kw, rc):
    assert _commit(lib, **kw) == rc


def test_no_device_after_the_checks(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _prompt(lib) == 5 and _prompt(lib, cu_k=None) == 5
    assert _tree(lib) == 5 and _tree(lib, N=64, kpos=A) == 5
    assert _logprobs(lib) == 5 and _logprobs(lib, lp=None, t=None) == 5
    assert _commit(lib) == 5 and _commit(lib, kpos=A, status=A) == 5


def test_binding_refuses_host_tensors():
    import torch
    import bit_weight_only_w4a16_gb300 as w4
    q = torch.zeros(4, 8, 256, dtype=torch.bfloat16)
    kv = torch.zeros(4, 1, 256, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.w4_attn_prompt(q, kv, kv, cu)
    with pytest.raises(ValueError):
        w4.w4_attn_tree(q[None], kv[None], kv[None], kv[None], kv[None], cu, cu)
    with pytest.raises(ValueError):
        w4.w4_logprobs(torch.zeros(2, 5))
    with pytest.raises(ValueError):
        c = torch.zeros(1, 1, 4, 8, dtype=torch.bfloat16)
        w4.w4_kv_commit(c, c, c, c, cu, cu, cu)

"""The serving calls' native binding: the same results as the Python one, and None (so that
the Python one makes the call or says what is wrong) for whatever is not plainly right."""
import numpy as np
import pytest
import torch

import bit_weight_only_w4a16_gb300 as w4

fast = w4._fast
pytestmark = pytest.mark.skipif(fast is None, reason="built without the native binding")


def on(where):
    """Arguments of each native call, in place."""
    def t(*s, dtype=torch.float32):
        return torch.zeros(s, dtype=dtype, device=where)

    i32, bf = torch.int32, torch.bfloat16
    q, k = t(4, 8, 64), t(4, 1, 64)
    pages = t(5, 16, 1, 64, dtype=bf)
    table, lens, cu = t(2, 3, dtype=i32), t(2, dtype=i32) + 5, torch.tensor([0, 2, 4], dtype=i32, device=where)
    table[1] += 1
    return {
        "lora": [t(4, 64), t(4, 32, dtype=bf), t(2, 8, 32, dtype=bf), t(2, 64, 8, dtype=bf), t(4, dtype=i32), t(2), None, None,
                 None],
        "rope": [q, k, t(4, dtype=i32), t(16), t(64), t(64), 1e-6, False, None, None, None],
        "qkv": [q, k, k, pages, pages, table, lens, t(16), cu, t(64), t(64), t(64), 1e-6, False, None, t(1, dtype=i32), None],
        "attn": [q.to(bf), pages, pages, table, lens, cu, 0, 1.0, None, None],
    }


CALLS = ["lora", "rope", "qkv", "attn"]


@pytest.mark.parametrize("call", CALLS)
def test_host_tensors_and_nonsense_are_left_to_python(call):
    f, args = getattr(fast, call), on("cpu")[call]
    assert f(*args) is None
    assert f() is None and f(*args, None) is None
    for i in range(len(args)):
        for bad in (None, "x", 7, object(), torch.zeros(1), 2.0 ** 70, 1 << 80):
            assert f(*(args[:i] + [bad] + args[i + 1:])) is None


class Sub(torch.Tensor):
    pass


PYTHON = {"lora": w4.w4_lora, "rope": w4.w4_qk_norm_rope, "qkv": w4.w4_qkv_paged, "attn": w4.w4_attn_paged}


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS)
def test_what_python_refuses_is_left_to_python(monkeypatch, call):
    """Every argument in other types, shapes, orders and places: what the native binding serves, the Python
    one serves with the same result."""
    w4.init()
    f, args = getattr(fast, call), on("cuda")[call]
    assert f(*args) is not None
    monkeypatch.setattr(w4, "_fast", None)
    served = left = 0
    for i, a in enumerate(args):
        if not isinstance(a, torch.Tensor):
            continue
        bad = [a.cpu(), a.to(torch.float64), a.to(torch.int64), a.unsqueeze(0).unsqueeze(0), torch.cat([a, a]), a.to_sparse(),
               a.as_subclass(Sub)]
        if a.shape[-1] > 1:
            bad += [torch.cat([a, a], -1)[..., ::2], a[..., :-1], a.flip(0)[..., :-1]]
        if a.dtype == torch.bfloat16:
            bad.append(a.view(torch.int16))  # raw bits: served, in Python
        for b in bad:
            those = args[:i] + [b] + args[i + 1:]
            r = f(*those)
            left += r is None
            if r is not None:
                served += 1
                want = PYTHON[call](*those)
                for u, v in zip(*((x,) if isinstance(x, torch.Tensor) else x for x in (r, want))):
                    assert torch.equal(u, v)
    assert left > 5 * served > 0
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_refusals_of_the_library_come_through():
    w4.init()
    a = on("cuda")
    y, x, la, lb, ids, s = a["lora"][:6]
    with pytest.raises(w4.W4Error, match="w4_lora -> W4_ERR_UNSUPPORTED"):
        w4.w4_lora(y, x, torch.cat([la[:, :4]] * 3, 1), torch.cat([lb[..., :4]] * 3, -1), ids)
    with pytest.raises(w4.W4Error, match="w4_qk_norm_rope -> W4_ERR_INVALID_ARG"):
        w4.w4_qk_norm_rope(*a["rope"][:4], eps=-1.0)
    with pytest.raises(w4.W4Error, match="w4_attn_paged -> W4_ERR_INVALID_ARG"):
        w4.w4_attn_paged(*a["attn"][:6], scale=0.0)
    with pytest.raises(w4.W4Error, match="w4_qkv_paged -> W4_ERR_UNSUPPORTED"):
        w4.w4_qkv_paged(*a["qkv"][:3], a["qkv"][3][:, :8], a["qkv"][4][:, :8], *a["qkv"][5:8], cu_q=a["qkv"][8])
    with pytest.raises(ValueError):
        w4.w4_qkv_paged(*a["qkv"][:6], a["qkv"][6][:1], a["qkv"][7])


def randn(g, *s, dtype=torch.float32):
    return torch.randn(*s, generator=g, device="cuda").to(dtype)


def both(monkeypatch, make):
    """make() through the native binding and through Python alone."""
    results = []
    for native in (True, False):
        with monkeypatch.context() as m:
            if not native:
                m.setattr(w4, "_fast", None)
            results.append(make())
    return results


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("other_stream", [False, True])
def test_the_same_results(monkeypatch, given, other_stream):
    w4.init()
    g = torch.Generator(device="cuda").manual_seed(1)
    M, Hq, Hkv, D, bf = 6, 8, 2, 128, torch.bfloat16
    wide = randn(g, M, (Hq + 2 * Hkv) * D + 8)
    q, k, v = (wide[:, i * D:j * D].view(M, j - i, D) for i, j in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    f, w = randn(g, 32).abs(), randn(g, D)
    x, la, lb = randn(g, M, 64, dtype=bf), randn(g, 3, 8, 64, dtype=bf), randn(g, 3, wide.shape[1], 8, dtype=bf)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, pos = torch.tensor([0, 2, -1, 1, 9, 0], **i32), torch.arange(M, **i32)
    table, lens, cu = torch.tensor([[3, 1], [0, 2]], **i32), torch.tensor([20, 3], **i32), torch.tensor([0, 4, 6], **i32)
    pools = [randn(g, 4, 2, 16, Hkv, D, dtype=bf) for _ in range(2)]
    stream = torch.cuda.Stream() if other_stream else None
    torch.cuda.synchronize()

    def run():
        kv = pools[0].clone()
        kp, vp = kv[:, 0], kv[:, 1]
        st = torch.zeros(2, **i32)
        o = [torch.full(s, 7.0, dtype=t, device="cuda") if given else None for s, t in
             (((M, wide.shape[1] + 8), torch.float32), ((M, Hq, D), bf), ((M, Hkv, D), bf), ((M, Hq, D), bf), ((M, Hq, D), bf))]
        torch.cuda.synchronize()
        z = w4.w4_lora(wide, x, la, lb, ids, scale=f[:3], out=None if o[0] is None else o[0][:, 8:], status=st[:1],
                       stream=stream)
        a, b = w4.w4_qk_norm_rope(q, k, pos, f, q_weight=w, eps=1e-5, pairs=True, q_out=o[1], k_out=o[2], stream=stream)
        c, none = w4.w4_qk_norm_rope(q.to(bf), None, pos, None, q_weight=w, stream=stream)
        d = w4.w4_qkv_paged(q, k, v, kp, vp, table, lens, f, cu_q=cu, v_weight=w, q_out=o[3], status=st[1:], stream=stream)
        e = w4.w4_attn_paged(d, kp, vp, table, lens, cu_q=cu, window=9, scale=0.1, out=o[4], stream=stream)
        h = w4.w4_attn_paged(d[:2], kp, vp, table, lens, scale=1, stream=stream)
        torch.cuda.synchronize()
        assert none is None
        if given:
            assert z.data_ptr() == o[0][:, 8:].data_ptr() and a is o[1] and b is o[2] and d is o[3] and e is o[4]
            assert bool((o[0][:, :8] == 7).all())
        assert all(t.dtype == (torch.float32 if t is z else bf) and not t.requires_grad for t in (z, a, b, c, d, e, h))
        return z, a, b, c, d, e, h, kv, st

    first, second = both(monkeypatch, run)
    for i, (u, t) in enumerate(zip(first, second)):
        assert torch.equal(u, t), i
    assert first[-1].tolist() == [1, 0]


@pytest.mark.gpu
def test_used_where_it_can_be(monkeypatch):
    """The usual call does not reach the Python checks."""
    w4.init()
    monkeypatch.setattr(w4, "_lib", None)
    a = on("cuda")
    assert w4.w4_lora(*a["lora"][:5]).shape == (4, 64)
    assert w4.w4_attn_paged(*a["attn"][:5], cu_q=a["attn"][5]).shape == (4, 8, 64)
    assert w4.w4_qk_norm_rope(*a["rope"][:4])[1].shape == (4, 1, 64)
    assert w4.w4_qkv_paged(*a["qkv"][:8], cu_q=a["qkv"][8]).shape == (4, 8, 64)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_no_reference_is_lost():
    """Outputs and arguments are counted as they are held."""
    import sys
    w4.init()
    a = on("cuda")
    out = torch.zeros(4, 64, device="cuda")
    args = a["lora"][:5]
    before = [sys.getrefcount(t) for t in args + [out]]
    for _ in range(20):
        w4.w4_lora(*args, out=out)
        w4.w4_qk_norm_rope(*a["rope"][:4])
    assert [sys.getrefcount(t) for t in args + [out]] == before
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    for _ in range(50):
        w4.w4_qk_norm_rope(*a["rope"][:4])
        w4.w4_attn_paged(*a["attn"][:5], cu_q=a["attn"][5])
        fast.lora(*a["lora"][:4], None, None, None, None, None)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == held
    assert np.isfinite(out.cpu().numpy()).all()

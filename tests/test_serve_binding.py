"""The serving calls refuse tensors that are not all on the current device and sizes past 32
bits (the C calls take 32-bit numbers). Shapes alone, no device memory."""
import pytest
import torch
from torch._subclasses import FakeTensorMode

import bit_weight_only_w4a16_gb300 as w4


class NoCalls:
    """In the library's place: no call may get through the checks."""

    def __getattr__(self, name):
        def called(*args):
            raise AssertionError(f"{name} was called")
        return called


def calls(where):
    """The calls with every tensor in its place; where(name) is a tensor's device."""
    def make(name, *s, dtype=torch.bfloat16):
        return torch.empty(s, dtype=dtype, device=where(name))

    def i32(name, *s):
        return make(name, *s, dtype=torch.int32)

    def f32(name, *s):
        return make(name, *s, dtype=torch.float32)

    def batch():
        return i32("table", 2, 3), i32("lens", 2)

    return {
        "rope": lambda: w4.w4_qk_norm_rope(f32("q", 4, 8, 64), f32("k", 4, 1, 64), i32("pos", 4), f32("inv_freq", 16),
                                           q_weight=f32("q_weight", 64), k_weight=f32("k_weight", 64),
                                           q_out=make("q_out", 4, 8, 64), k_out=make("k_out", 4, 1, 64)),
        "qkv": lambda: w4.w4_qkv_paged(f32("q", 4, 8, 64), f32("k", 4, 1, 64), f32("v", 4, 1, 64),
                                       make("k_pages", 5, 16, 1, 64), make("v_pages", 5, 16, 1, 64), *batch(),
                                       f32("inv_freq", 16), cu_q=i32("cu_q", 3), q_weight=f32("q_weight", 64),
                                       k_weight=f32("k_weight", 64), v_weight=f32("v_weight", 64),
                                       q_out=make("q_out", 4, 8, 64), status=i32("status", 1)),
        "attn": lambda: w4.w4_attn_paged(make("q", 4, 8, 64), make("k_pages", 5, 16, 1, 64), make("v_pages", 5, 16, 1, 64),
                                         *batch(), cu_q=i32("cu_q", 3), out=make("out", 4, 8, 64)),
        "lora": lambda: w4.w4_lora(f32("y", 4, 64), make("x", 4, 32), make("a", 2, 8, 32), make("b", 2, 64, 8), i32("ids", 4),
                                   scale=f32("scale", 2), out=f32("out", 4, 64), status=i32("status", 1)),
    }


TENSORS = {
    "rope": ["q", "k", "pos", "inv_freq", "q_weight", "k_weight", "q_out", "k_out"],
    "qkv": ["q", "k", "v", "k_pages", "v_pages", "table", "lens", "inv_freq", "cu_q", "q_weight", "k_weight", "v_weight",
            "q_out", "status"],
    "attn": ["q", "k_pages", "v_pages", "table", "lens", "cu_q", "out"],
    "lora": ["y", "x", "a", "b", "ids", "scale", "out", "status"],
}


@pytest.mark.parametrize("call,odd", [(c, t) for c, ts in TENSORS.items() for t in ts])
@pytest.mark.parametrize("other", ["cuda:1", "cpu"])
def test_one_tensor_elsewhere(monkeypatch, call, odd, other):
    monkeypatch.setattr(w4, "_current_device", lambda: 0)
    monkeypatch.setattr(w4, "_lib", NoCalls())
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 1 << 20)
    with FakeTensorMode():
        with pytest.raises(ValueError, match="device|CUDA"):
            calls(lambda name: other if name == odd else "cuda:0")[call]()


@pytest.mark.parametrize("call", list(TENSORS))
def test_all_on_another_device_than_the_current_one(monkeypatch, call):
    monkeypatch.setattr(w4, "_current_device", lambda: 0)
    with FakeTensorMode():
        with pytest.raises(ValueError, match="current device is 0"):
            calls(lambda name: "cuda:1")[call]()


P = 2 ** 32


@pytest.fixture
def make(monkeypatch):
    monkeypatch.setattr(w4, "_current_device", lambda: 0)
    monkeypatch.setattr(w4, "_lib", NoCalls())
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 1 << 20)
    with FakeTensorMode():
        yield lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda:0")


@pytest.mark.parametrize("M", [P + 2, 2 ** 31])
def test_rows_past_32_bits(make, M):
    i32 = lambda *s: make(*s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: make(*s, dtype=torch.float32)  # noqa: E731
    pool = make(5, 16, 1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_qk_norm_rope(make(M, 8, 64), make(M, 1, 64), i32(M), f32(32))
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_qkv_paged(make(M, 8, 64), make(M, 1, 64), make(M, 1, 64), pool, pool, i32(2, 3), i32(2), f32(32), cu_q=i32(3))
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_attn_paged(make(M, 8, 64), pool, pool, i32(2, 3), i32(2), cu_q=i32(3))
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_lora(f32(M, 64), make(M, 32), make(2, 8, 32), make(2, 64, 8), i32(M))


@pytest.mark.parametrize("window", [P, P + 7, 2 ** 31, -2 ** 31 - 1])
def test_windows_past_32_bits(make, window):
    i32 = lambda *s: make(*s, dtype=torch.int32)  # noqa: E731
    pool = make(5, 16, 1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_attn_paged(make(4, 8, 64), pool, pool, i32(2, 3), i32(2), cu_q=i32(3), window=window)


@pytest.mark.parametrize("n", [P + 1, 2 ** 31])
def test_pools_tables_and_adapters_past_32_bits(make, n):
    i32 = lambda *s: make(*s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: make(*s, dtype=torch.float32)  # noqa: E731
    big, pool = make(n, 16, 1, 64), make(5, 16, 1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_attn_paged(make(4, 8, 64), big, big, i32(2, 3), i32(2), cu_q=i32(3))
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_attn_paged(make(4, 8, 64), pool, pool, i32(2, n), i32(2), cu_q=i32(3))
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_qkv_paged(make(2, 8, 64), make(2, 1, 64), make(2, 1, 64), pool, pool, i32(2, n), i32(2), f32(32))
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_lora(f32(4, 64), make(4, 32), make(n, 8, 32), make(n, 64, 8), i32(4))

"""The native binding where the library's call fails.

The library's functions are replaced by stand-ins, so nothing is launched."""
import ctypes

import pytest
import torch

import bit_weight_only_w4a16_gb300 as w4

fast = w4._fast
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(fast is None, reason="built without the native binding")]

NAMES = ("w4_lora", "w4_qk_norm_rope", "w4_qkv_paged", "w4_attn_paged")


def address(f):
    return ctypes.cast(f, ctypes.c_void_p).value


@pytest.fixture
def bound():
    """fast.bind for the length of a test."""
    w4.init()
    own = [address(getattr(w4._lib, n)) for n in NAMES]
    yield lambda f: fast.bind(*[address(f)] * 4)
    fast.bind(*own)


def calls():
    def t(*s, dtype=torch.float32):
        return torch.zeros(s, dtype=dtype, device="cuda")

    i32, bf = torch.int32, torch.bfloat16
    q, k, pages = t(2, 8, 64), t(2, 1, 64), t(5, 16, 1, 64, dtype=bf)
    table, lens = t(2, 3, dtype=i32), t(2, dtype=i32) + 5
    return {
        "w4_lora": lambda: w4.w4_lora(t(4, 64), t(4, 32, dtype=bf), t(2, 8, 32, dtype=bf), t(2, 64, 8, dtype=bf),
                                      t(4, dtype=i32)),
        "w4_qk_norm_rope": lambda: w4.w4_qk_norm_rope(q, k, t(2, dtype=i32), t(16)),
        "w4_qkv_paged": lambda: w4.w4_qkv_paged(q, k, k, pages, pages, table, lens, t(16)),
        "w4_attn_paged": lambda: w4.w4_attn_paged(q.to(bf), pages, pages, table, lens),
    }


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("status,again", [(1, 1), (2, 1), (3, 1), (4, 0), (5, 0)])
def test_a_failed_launch_is_not_repeated(monkeypatch, bound, name, status, again):
    """Refused arguments (1 to 3) launched nothing: the Python binding says what is wrong. A call that failed
    later may have done a part of its work, in place: it is not made a second time."""
    made = {"native": 0, "python": 0}

    @ctypes.CFUNCTYPE(ctypes.c_int)
    def failing():
        made["native"] += 1
        return status

    class Library:
        def __getattr__(self, n):
            if n not in NAMES:
                return getattr(real, n)

            def call(*args):
                made["python"] += 1
                return status
            return call

    call, real = calls()[name], w4._lib
    monkeypatch.setattr(w4, "_lib", Library())
    bound(failing)
    with pytest.raises(w4.W4Error, match=f"{name} -> ") as e:
        call()
    assert e.value.status == status
    assert made == {"native": 1, "python": again}

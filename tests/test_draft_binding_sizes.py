"""Sizes and windows past 32 bits are refused by the binding, whose C calls take 32-bit
numbers (they would be cut to their low bits). Shapes alone, no device memory."""
import pytest
import torch
from torch._subclasses import FakeTensorMode

import bit_weight_only_w4a16_gb300 as w4

P = 2 ** 32


@pytest.fixture
def make():
    with FakeTensorMode():
        yield lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")


@pytest.mark.parametrize("M,V,k", [(1, P + 5, 0), (1, 2 ** 31, 0), (P + 1, 3, 0), (2, 10, P + 1)])
def test_logprobs(make, M, V, k):
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_logprobs(make(M, V, dtype=torch.float32), topk=k)


@pytest.mark.parametrize("window", [P, P + 7, 2 ** 31, -P + 7, -2 ** 31 - 1])
def test_windows(make, window):
    i32 = lambda *s: make(*s, dtype=torch.int32)  # noqa: E731
    q, kv = make(4, 8, 64), make(4, 1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_attn_prompt(q, kv, kv, i32(2), window=window)
    c = make(1, 16, 1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_attn_tree(q[None], c, c, kv[None], kv[None], i32(1, 4), i32(1), window=window)


@pytest.mark.parametrize("rows", [P + 4, 2 ** 31])
def test_attention_rows(make, rows):
    i32 = lambda *s: make(*s, dtype=torch.int32)  # noqa: E731
    q, kv = make(4, 8, 64), make(4, 1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_attn_prompt(q, make(rows, 1, 64), make(rows, 1, 64), i32(2))
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_attn_prompt(make(rows, 1, 64), kv, kv, i32(2))
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_attn_tree(q[None], make(1, rows, 1, 64), make(1, rows, 1, 64), kv[None], kv[None], i32(1, 4), i32(1))


@pytest.mark.parametrize("shape", [(1, 1, P + 16, 8), (P + 1, 1, 16, 8), (1, 1, 16, P + 8)])
def test_commit(make, shape):
    i32 = lambda *s: make(*s, dtype=torch.int32)  # noqa: E731
    L, B, T, W = shape
    c, t = make(*shape), make(L, B, 4, W)
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_kv_commit(c, c, t, t, i32(B, 4), i32(B), i32(B))

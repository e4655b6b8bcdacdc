"""Calls in which one CTA works on one row tile for a second: what waits for a whole row
tile waits longer than the steps within it do.

Queries of zeros weigh every key alike and values of 0 and +-1 sum to whole numbers of a
few thousand, exact in fp32; the division and the rounding to bf16 (2^-8) are left.
"""
import pytest

from test_attn_prompt_parity import w4  # noqa: F401

pytestmark = pytest.mark.gpu


def test_row_tiles_of_a_second(w4):  # noqa: F811
    """As many row tiles as SMs over 80 million keys (keys and values are one tensor)."""
    import torch
    rows = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    lk, D, G = 80_000_000, 64, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(0, 32, (lk, 1, D), generator=g, device="cuda", dtype=torch.int8)
    kv = (x == 0).to(torch.bfloat16) - (x == 1).to(torch.bfloat16)
    del x
    q = torch.zeros(rows, G, D, dtype=torch.bfloat16, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = w4.w4_attn_prompt(q, kv, kv, i32([0, rows]), i32([0, lk]), scale=0.1)
    assert w4.device_error() == 0
    first = lk - rows
    sums = kv[:first, 0].sum(0, dtype=torch.float64) + kv[first:, 0].double().cumsum(0)
    want = (sums / torch.arange(first + 1, lk + 1, device="cuda")[:, None])[:, None].expand(rows, G, D)
    assert bool(((out.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -20)).all())

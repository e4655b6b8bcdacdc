"""The example's shortest prompts: one token (nothing to read before the first step) and two."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length", [1, 2])
def test_prompt(length):
    import torch

    import bit_weight_only_w4a16_gb300 as w4
    from examples import draft_step as ex
    w4.init()
    prompt = torch.tensor([5, 17][:length], dtype=torch.int32, device="cuda")
    plain, lp, steps = ex.decode(ex.Model(), prompt, 12, ex.no_draft)
    assert steps == 12 and len(plain) == 12
    drafted, _, fewer = ex.decode(ex.Model(), prompt, 12, ex.TruthDraft(length, plain, 2048))
    assert drafted == plain and fewer < steps

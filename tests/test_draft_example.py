"""examples/draft_step.py: decoding with drafted trees gives the tokens of plain
decoding in fewer steps, past the ring's wrap."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_drafted_decoding_equals_plain():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import draft_step
    same, steps, drafted = draft_step.main(prompt_len=130, n=40)
    assert same and steps == 40 and drafted <= 25

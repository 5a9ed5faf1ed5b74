"""The draft operators together, as a serving loop uses them: a head that is
distilled from the verified target's logits comes to have more of its drafts
accepted."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_a_learning_head_gets_more_drafts_accepted():
    import online_draft_head
    first, final, losses = online_draft_head.run(rounds=120, report=lambda *_: None)
    assert losses[-1] < 0.5 * losses[0]
    assert final > first + 0.3

"""examples/online_distill.py: accept, scores and distillation together, as a serving loop
that trains its drafter would run them."""
import os
import sys

import pytest

from libs import ROOT, ensure_built

pytestmark = pytest.mark.gpu


def test_the_drafter_learns_from_the_target():
    ensure_built()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import online_distill
    history = online_distill.train(rounds=160)
    first, last = history[:10], history[-10:]
    mean = lambda rows, i: sum(r[i] for r in rows) / len(rows)  # noqa: E731
    assert mean(last, 1) < 0.5 * mean(first, 1)  # the loss
    assert mean(last, 0) > mean(first, 0) + 0.5  # drafts accepted a round
    assert all(-5.0 < r[2] < 0.0 for r in history)

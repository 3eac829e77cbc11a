"""The operators and the optimizer step together: a small tied-table model learns.

The text repeats 7 of 8 words, so the loss starts at ln(500) = 6.2 for even odds
and its floor is near 1/8 ln(500 * 8) + 7/8 ln(8/7) = 1.15.  A step that lost a
gradient, a sign or a scale of the table's two gradients does not come below half
of the start."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_tied_model_learns():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import tied_lm
    losses, norms = tied_lm.train(steps=120)
    assert 5.0 < losses[0] < 9.0
    assert min(losses[-5:]) < 0.5 * losses[0]
    assert all(0.0 < n < 1e4 for n in norms)

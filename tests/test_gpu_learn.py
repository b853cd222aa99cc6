"""The learning study: recurrence, solves, adjoints and AdamW steps together."""
import numpy as np
import pytest

from preconditioned_cg_solver_amd import studies
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_rates_and_strengths_are_learnt(bits):
    """The data are exact, so the loss has a zero that the parameters reach: in
    80 steps of at most 0.05 (the parameters start within about 1.5 of it) the
    loss falls by two decades, and the strengths, which every observed field
    shows directly, come within a tenth of their spread."""
    say("learn", bits)
    out = studies.learn(iters=80, bits=bits)
    assert np.isfinite(out["loss_last"])
    assert out["loss_last"] <= 1e-2 * out["loss_first"], out
    assert out["strength_error"] <= 0.1 and out["rate_error"] < 0.7, out

"""What the C entry points of a sequence block's operators refuse at their edges (no GPU)."""
import ctypes

import pytest

from preconditioned_cg_solver_amd import binding as B
from test_block_host import INVALID, L, P, conv_backward, conv_shape  # noqa: F401


@pytest.mark.parametrize("bad", [dict(dx=None), dict(dx=P[0]), dict(dx=P[4]), dict(dw=None)])
def test_conv_without_a_sequence_refuses(L, bad):  # noqa: F811
    """Packed rows without a sequence have gradients to be written, and somewhere to be."""
    q = conv_shape(n_seq=0, steps=70, d_offsets=P[12])
    assert conv_backward(L, q, **bad) == INVALID
    assert L.sla_last_error()

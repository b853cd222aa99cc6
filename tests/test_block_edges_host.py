"""What the C entry points of a sequence block's operators refuse at their edges (no GPU)."""
import pytest

from preconditioned_cg_solver_amd import binding as B
from test_block_host import (INVALID, L, P, conv_backward, conv_shape, scan_backward,  # noqa: F401
                             scan_in, scan_shape)


@pytest.mark.parametrize("bad", [dict(dx=None), dict(dx=P[0]), dict(dx=P[4]), dict(dw=None)])
def test_conv_without_a_sequence_refuses(L, bad):  # noqa: F811
    """Packed rows without a sequence have gradients to be written, and somewhere to be."""
    q = conv_shape(n_seq=0, steps=70, d_offsets=P[12])
    assert conv_backward(L, q, **bad) == INVALID
    assert L.sla_last_error()


@pytest.mark.parametrize("bad", [dict(d_x=None), dict(d_dt=None), dict(d_z=None), dict(d_b=None),
                                 dict(d_c=None), dict(d_a=None), dict(d_x=P[0]), dict(d_b=P[4]),
                                 dict(d_b=P[16])])
def test_scan_without_a_sequence_refuses(L, bad):  # noqa: F811
    q = scan_shape(n_seq=0, steps=70, d_offsets=P[21])
    assert scan_backward(L, q, scan_in(), saved=None, **bad) == INVALID
    assert L.sla_last_error()

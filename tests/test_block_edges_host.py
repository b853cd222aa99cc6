"""What the C entry points of a sequence block's operators refuse at their edges (no GPU)."""
import itertools

import pytest

from preconditioned_cg_solver_amd import binding as B
from test_block_host import (INVALID, L, OK, P, conv_backward, conv_shape, norm_shape,  # noqa: F401
                             norm_sizes, scan_backward, scan_in, scan_shape)


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


def test_norm_workspace_holds_the_parts_that_there_are(L):  # noqa: F811
    """Two rows of sums for each team of waves: 4096 teams of one wave for rows that a wave reads at
    once, 1024 of several for wider ones, 512 of sixteen; never more than there are rows to take."""
    for dtype, size in ((B.SLA_BF16, 2), (B.SLA_F32, 4), (B.SLA_F64, 8)):
        own = 8 if size == 8 else 4
        for rows, dim in itertools.product((1, 3, 100, 5000, 1 << 20), (8, 512, 2048, 4104, 1 << 20)):
            q = norm_shape(rows=rows, dim=dim, dtype=dtype, stream=dtype)
            st, n = norm_sizes(L, q)
            least = 4096 if dim * size <= 1024 else 1024 if dim * size <= 8192 or dim <= 1024 else 512
            teams = min(-(-rows // 4) * 4 if least == 4096 else rows, least)
            assert st == OK and n == -(-teams * 2 * dim * own // 256) * 256, (dtype, rows, dim)

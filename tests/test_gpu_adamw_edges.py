"""Edges of the AdamW step: values that are not finite, steps that go past the
caches, memory shared with other tensors and streams."""
import pytest
import torch

from preconditioned_cg_solver_amd import binding as B
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float64, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_second_moment_that_is_not_a_number(dtype, bits):
    """beta2 = 0 makes a NaN of an infinite v, and a NaN divides the update: the
    formula's parameter is a NaN, in its own element alone."""
    say("adamw NaN in v", dtype, bits)
    n = 600
    p, q = (torch.ones(n, device=DEV, dtype=dtype) for _ in range(2))
    g = torch.full((n,), 0.5, device=DEV, dtype=dtype)
    a, b = (B.sla_adamw_create([t], state_bits=bits) for t in (p, q))
    m = torch.full((a.padded,), 0.25, device=DEV)
    m[n:] = 0.0
    v = m.clone()
    B.sla_adamw_set_state(b, m, v)
    v[7], v[300] = float("inf"), float("inf")
    B.sla_adamw_set_state(a, m, v)
    for opt in (a, b):
        B.sla_adamw_step(opt, [g], step=3, lr=1e-2, beta2=0.0, seed=1)
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[7] = bad[300] = True
    assert torch.equal(torch.isnan(p), bad) and torch.equal(p[~bad], q[~bad])
    vs = B.sla_adamw_get_state(a)[1][:n]
    assert not bool(torch.isfinite(vs[bad]).any())

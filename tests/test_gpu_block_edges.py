"""Edges of a sequence block's operators on the GPU: batches of rows without a sequence, and
values that are not finite beside rows of no sequence."""
import pytest
import torch

from preconditioned_cg_solver_amd import autograd as AG
from preconditioned_cg_solver_amd import binding as B
from block_gpu import DT, make
from gpu_util import say

pytestmark = pytest.mark.gpu
SCAN = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")


def soil(*shapes, dtype):
    """Memory that is handed out again soon holds NaN."""
    held = [torch.full(s, float("nan"), dtype=dtype, device="cuda") for s in shapes for _ in range(6)]
    del held


def none_of(mark):
    return torch.tensor([mark], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [23, 512])
@pytest.mark.parametrize("mark", [0, 7, 70])
def test_conv_gradients_without_a_sequence(dtype, d, mark):
    """Offsets of one entry: all rows are of no sequence, and their gradients are zeros."""
    say("conv, no sequence", dtype, d, mark)
    r, off = make(0, dtype), none_of(mark)
    x, w, b, dy = r(70, d), r.own(d, 4), r.own(d), r(70, d)
    soil((70, d), dtype=DT[dtype])
    dx, dw, db, _ = B.sla_conv_backward(x, w, dy, bias=b, offsets=off)
    assert not dx.any() and not dw.any() and not db.any()
    x.requires_grad_(), w.requires_grad_()
    y, last = AG.causal_conv(x, w, b, offsets=off)
    assert not y.any() and last.shape == (0, 3, d)
    soil((70, d), dtype=DT[dtype])
    dx, dw = torch.autograd.grad(y.sum(), [x, w])
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d,N,groups", [(24, 16, 1), (23, 3, 1), (24, 4, 3)])
@pytest.mark.parametrize("mark", [0, 7, 70])
def test_scan_gradients_without_a_sequence(dtype, d, N, groups, mark):
    """Offsets of one entry: all rows are of no sequence, and their gradients are zeros."""
    say("scan, no sequence", dtype, d, N, groups, mark)
    r, off = make(1, dtype), none_of(mark)
    x, dt, z, dy = r(70, d), r(70, d), r(70, d), r(70, d)
    b, c = r(70, groups, N), r(70, groups, N)
    A, D, bias = -r.own(d, N).abs(), r.own(d), r.own(d)
    own = dict(D=D, z=z, dt_bias=bias, offsets=off)
    _, _, saved = B.sla_selscan_forward(x, dt, A, b, c, **own, save=True)
    soil((70, d), (70, groups, N), dtype=DT[dtype])
    grads = B.sla_selscan_backward(x, dt, A, b, c, saved, dy, **own)
    for name, g in zip(SCAN[:-1], grads):
        assert not g.any(), name
    leaves = [t.requires_grad_() for t in (x, dt, A, b, c, D, z, bias)]
    y, last = AG.selective_scan(x, dt, A, b, c, D=D, z=z, dt_bias=bias, offsets=off)
    assert not y.any() and last.shape == (0, d, N)
    soil((70, d), (70, groups, N), dtype=DT[dtype])
    for name, g in zip(SCAN[:-1], torch.autograd.grad(y.sum(), leaves)):
        assert not g.any(), name


@pytest.mark.parametrize("before,behind", [(37, 50), (5, 3), (200, 130)])
@pytest.mark.parametrize("d,N", [(24, 16), (23, 3)])
@pytest.mark.parametrize("what", ["gradient", "state", "rate"])
def test_padded_rows_beside_what_is_not_finite(what, d, N, before, behind):
    """An infinite gradient at the first row of the first sequence, an infinite state at the last
    of the last, a rate of -infinity: rows before and behind, which hold NaN, have gradients of
    zero, and the other results are those without such rows."""
    say("scan, not finite beside padding", what, d, N, before, behind)
    r = make(2, "f32")
    n, off = 50, torch.tensor([0, 20, 50], device="cuda")
    a = dict(x=r(n, d), dt=r(n, d), B=r(n, 1, N), C=r(n, 1, N), z=r(n, d))
    own = dict(D=r.own(d), dt_bias=r.own(d) - 2, h0=r.own(2, d, N))
    A, dy, dl = -r.own(d, N).abs(), r(n, d), r.own(2, d, N)
    if what == "gradient":
        dy[0, 3] = float("inf")
    elif what == "state":
        a["x"][-1, 5] = float("inf")
    else:
        A[7, 2] = float("-inf")

    def pad(t):
        return torch.cat([t.new_full((before, *t.shape[1:]), float("nan")), t,
                          t.new_full((behind, *t.shape[1:]), float("nan"))])

    def grads(a, off, dy):
        first = (a["x"], a["dt"], A, a["B"], a["C"])
        y, last, saved = B.sla_selscan_forward(*first, z=a["z"], **own, offsets=off, save=True)
        g = B.sla_selscan_backward(*first, saved, dy, grad_last=dl, z=a["z"], **own, offsets=off)
        return {"y": y, "last": last, **dict(zip(SCAN, g))}

    plain = grads(a, off, dy)
    padded = grads({k: pad(v) for k, v in a.items()}, off + before, pad(dy))
    for k, g in plain.items():
        p = padded[k]
        if g.shape[0] == n:
            rest = torch.cat([p[:before], p[before + n:]])
            assert (rest == 0).all(), k  # NaN is not 0
            p = p[before:before + n]
        # tiles and chunks lie elsewhere: equal to fp32 rounding, and as finite
        assert torch.equal(torch.isfinite(p), torch.isfinite(g)), k
        assert torch.allclose(p, g, rtol=1e-4, atol=1e-3, equal_nan=True), k

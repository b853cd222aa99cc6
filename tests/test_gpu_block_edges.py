"""Edges of a sequence block's operators on the GPU: batches of rows without a sequence, values that
are not finite beside rows of no sequence, and scans long or wide enough not to be cut."""
import pytest
import torch

from preconditioned_cg_solver_amd import autograd as AG
from preconditioned_cg_solver_amd import binding as B
import block_util as K
from block_gpu import DT, check, make, np64, offsets_of, unit_of
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


def scan_part(a, off, dy, dl, store, pick):
    """The reference of some channels, or sequences, of a call."""
    q = {k: v if v is None else np64(pick(k, v)) for k, v in {**a, "dy": dy, "dlast": dl}.items()}
    return K.scan(**q, offsets=off, unit=unit_of(store), store=store)


@pytest.mark.parametrize("dtype,d", [("bf16", 192), ("f32", 190), ("f64", 192)])
def test_long_scans_that_are_not_cut(dtype, d):
    """Enough sequences that each is one chunk in both directions (12 waves of channels each), of
    17 tiles and a part of one: three of them against the reference, the others without gradients so
    that the sums over all are sums over the three."""
    say("scan, long and uncut", dtype, d)
    r, n, steps, N = make(3, dtype), 128, 277, 16
    a = dict(x=r(n, steps, d), dt=r(n, steps, d), A=-r.own(d, N).abs(), B=r(n, steps, 1, N),
             C=r(n, steps, 1, N), D=r.own(d), z=r(n, steps, d), bias=r.own(d) - 2, h0=r.own(n, d, N))
    dy, dl = r(n, steps, d), r.own(n, d, N)
    some = [0, 77, 127]
    others = [s for s in range(n) if s not in some]
    dy[others], dl[others] = 0, 0
    kw = dict(D=a["D"], z=a["z"], dt_bias=a["bias"], h0=a["h0"])
    first = (a["x"], a["dt"], a["A"], a["B"], a["C"])
    assert B.sla_selscan_sizes(*first, **kw)[1] == 0  # nothing to join
    y, last, saved = B.sla_selscan_forward(*first, **kw, save=True)
    got = dict(zip(SCAN, B.sla_selscan_backward(*first, saved, dy, grad_last=dl, **kw)))
    got.update(y=y, last=last)
    whole = ("A", "D", "bias")
    want = scan_part(a, None, dy, dl, dtype, lambda k, v: v if k in whole else v[some])
    check({k: v if k[1:] in whole else v[some] for k, v in got.items()}, want)
    for k in ("dx", "ddt", "dB", "dC", "dz", "dh0"):
        assert not got[k][others].any(), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wide_packed_scans_that_are_not_cut(dtype):
    """Enough channels that packed sequences are one chunk: the first and the last of 64 groups
    against the reference."""
    say("scan, wide, packed and uncut", dtype)
    r, d, G, N, lengths = make(4, dtype), 24576, 64, 16, [40, 0, 3, 107]
    steps, per = sum(lengths), d // G
    off, n = offsets_of(lengths, (steps,))
    a = dict(x=r(steps, d), dt=r(steps, d), A=-r.own(d, N).abs(), B=r(steps, G, N),
             C=r(steps, G, N), D=r.own(d), z=r(steps, d), bias=r.own(d) - 2, h0=r.own(n, d, N))
    dy, dl = r(steps, d), r.own(n, d, N)
    kw = dict(D=a["D"], z=a["z"], dt_bias=a["bias"], h0=a["h0"], offsets=off)
    first = (a["x"], a["dt"], a["A"], a["B"], a["C"])
    assert B.sla_selscan_sizes(*first, **kw)[1] == 0  # nothing to join
    y, last, saved = B.sla_selscan_forward(*first, **kw, save=True)
    got = dict(zip(SCAN, B.sla_selscan_backward(*first, saved, dy, grad_last=dl, **kw)))
    got.update(y=y, last=last)
    for g in (0, G - 1):
        c = slice(g * per, (g + 1) * per)

        def pick(k, v):
            if k in ("A", "D", "bias", "dA", "dD", "dbias"):
                return v[c]
            return v[:, g:g + 1] if k in ("B", "C", "dB", "dC") else v[:, c]

        want = scan_part(a, np64(off).astype(int), dy, dl, dtype, pick)
        check({k: pick(k, v) for k, v in got.items()}, want)

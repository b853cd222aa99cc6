"""Causal convolutions on the GPU against the 64-bit reference and its error bounds."""
import numpy as np
import pytest
import torch

from preconditioned_cg_solver_amd import binding as B
import block_util as K
from block_gpu import DT, check, make, np64, offsets_of, own_of, unit_of
from gpu_util import say

pytestmark = pytest.mark.gpu


def run(dtype, lead, d, k, act="silu", lengths=None, state=True, bias=True, strided=False,
        grads=True, seed=0):
    say("conv", dtype, lead, d, k, act, lengths, state, bias, strided)
    r = make(seed, dtype)
    off, n = offsets_of(lengths, lead)
    x = r(*lead, d, strided=strided)
    w, b = r.own(d, k), r.own(d) if bias else None
    st = r(n, k - 1, d) if state else None
    y, last = B.sla_conv_forward(x, w, bias=b, state=st, offsets=off, act=act)
    got = {"y": y, "last": last}
    dy = dl = None
    if grads:
        dy, dl = r(*lead, d, strided=strided), r(n, k - 1, d)
        got["dx"], got["dw"], got["db"], got["dstate"] = B.sla_conv_backward(
            x, w, dy, bias=b, state=st, grad_last=dl, offsets=off, act=act)
    want = K.conv(*map(np64, (x, w, b, st)), None if off is None else np64(off).astype(int), act,
                  np64(dy), np64(dl), unit=unit_of(dtype), store=dtype)
    check(got, want)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("k", [2, 3, 4])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_types_taps_activations(dtype, k, act):
    run(dtype, (2, 37), 72, k, act)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7, 8, 9, 16, 17, 130])
@pytest.mark.parametrize("d", [1, 5, 64, 260])
def test_lengths_and_widths(steps, d):
    run("bf16", (3, steps), d, 4)
    run("f32", (1, steps), d, 3, state=False)


@pytest.mark.parametrize("lengths", [[0, 1, 2, 3, 0, 40, 9], [5], [1] * 12, [0, 0, 17], [33, 0, 0],
                                     [3] + [0] * 9 + [20]])
@pytest.mark.parametrize("d", [3, 256])
@pytest.mark.parametrize("k", [2, 4])
def test_packed(lengths, d, k):
    run("f16", (sum(lengths),), d, k, lengths=lengths)
    run("f32", (sum(lengths),), d, k, lengths=lengths, state=False, bias=False)


@pytest.mark.parametrize("dtype", list(DT))
def test_slices_of_wider_tensors(dtype):
    run(dtype, (2, 19), 512, 4, strided=True)
    run(dtype, (50,), 33, 3, lengths=[20, 30], strided=True)


def test_several_runs_of_steps():
    run("bf16", (1, 600), 1024, 4)
    run("f32", (700,), 130, 4, lengths=[1, 300, 2, 397])


def test_no_steps():
    r = make(1, "f32")
    x, w, st, dl = r(2, 0, 5), r.own(5, 4), r(2, 3, 5), r(2, 3, 5)
    y, last = B.sla_conv_forward(x, w, state=st)
    assert y.shape == x.shape and torch.equal(last, st)
    dx, dw, _, dst = B.sla_conv_backward(x, w, x, state=st, grad_last=dl)
    assert dx.numel() == 0 and not dw.any() and torch.equal(dst, dl)
    _, last = B.sla_conv_forward(x, w)
    assert not last.any()
    y, last = B.sla_conv_forward(r(0, 4, 5), w)
    assert y.shape == (0, 4, 5) and last.shape == (0, 3, 5)
    dx, dw, _, _ = B.sla_conv_backward(r(0, 4, 5), w, r(0, 4, 5))
    assert not dw.any()


@pytest.mark.parametrize("steps", [1, 5, 300])
@pytest.mark.parametrize("packed", [False, True])
def test_state_updated_in_place(steps, packed):
    r = make(2, "bf16")
    n, d = 3, 192
    lead = (n * steps,) if packed else (n, steps)
    off = torch.arange(n + 1, device="cuda") * steps if packed else None
    x, w, st = r(*lead, d), r.own(d, 4), r(n, 3, d)
    y, last = B.sla_conv_forward(x, w, state=st, offsets=off)
    held = st.clone()
    y2, last2 = B.sla_conv_forward(x, w, state=held, offsets=off, last=held)
    assert last2 is held and torch.equal(y, y2) and torch.equal(last, held)


def test_steps_one_by_one_are_the_whole():
    r = make(3, "bf16")
    x, w, b = r(2, 21, 96), r.own(96, 4), r.own(96)
    whole, last = B.sla_conv_forward(x, w, bias=b)
    st = torch.zeros(2, 3, 96, device="cuda", dtype=x.dtype)
    parts = [B.sla_conv_forward(x[:, t:t + 1], w, bias=b, state=st, last=st)[0] for t in range(21)]
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(st, last)


def test_values_that_are_not_finite_stay_in_their_reach():
    """A channel's infinite or undefined input reaches the outputs of its own taps only;
    -infinity before the activation gives 0."""
    r = make(4, "f32")
    x, w = r(2, 40, 8), r.own(8, 4).abs()
    y0, _ = B.sla_conv_forward(x, w)
    for v in (float("nan"), float("inf"), float("-inf")):
        bad = x.clone()
        bad[1, 10, 3] = v
        y, _ = B.sla_conv_forward(bad, w)
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[1, 10:14, 3] = True
        assert torch.equal(y[~hit], y0[~hit])
        if v == float("-inf"):
            assert (y[hit] == 0).all()
        else:
            assert not torch.isfinite(y[hit]).any()


@pytest.mark.parametrize("before,behind", [(0, 40), (5, 0), (17, 133)])
@pytest.mark.parametrize("d", [3, 512])
def test_padded_rows_are_of_no_sequence(before, behind, d):
    """Rows before the first and behind the last sequence hold NaN: the results are those without
    them, the weights' gradients too, and their own gradients are zeros."""
    r = make(11, "bf16")
    lengths = [30, 0, 2, 100, 1]
    n = sum(lengths)
    off, _ = offsets_of(lengths, (n,))
    x, w, b, st = r(n, d), r.own(d, 4), r.own(d), r(5, 3, d)
    dy, dl = r(n, d), r(5, 3, d)

    def pad(t):
        return torch.cat([t.new_full((before, d), float("nan")), t,
                          t.new_full((behind, d), float("nan"))])

    y, last = B.sla_conv_forward(x, w, bias=b, state=st, offsets=off)
    g = B.sla_conv_backward(x, w, dy, bias=b, state=st, grad_last=dl, offsets=off)
    py, plast = B.sla_conv_forward(pad(x), w, bias=b, state=st, offsets=off + before)
    pg = B.sla_conv_backward(pad(x), w, pad(dy), bias=b, state=st, grad_last=dl,
                             offsets=off + before)
    assert torch.equal(py[before:before + n], y) and torch.equal(plast, last)
    assert torch.equal(pg[0][before:before + n], g[0]) and torch.equal(pg[3], g[3])
    assert not pg[0][:before].any() and not pg[0][before + n:].any()
    assert torch.allclose(pg[1], g[1], rtol=1e-4, atol=1e-4)  # other runs, other order
    assert torch.allclose(pg[2], g[2], rtol=1e-4, atol=1e-4)


def test_arbitrary_offsets_leave_the_neighbours_alone():
    """Offsets that do not ascend give some result, within the arrays."""
    d, n, steps = 64, 5, 50
    big = torch.full((steps + 200, d), 7.0, device="cuda")
    off = torch.tensor([40, -3, 900, 12, 12, -70], device="cuda")
    x, w, st = big[100:100 + steps], torch.ones(d, 4, device="cuda"), torch.ones(n, 3, d, device="cuda")
    y, last = B.sla_conv_forward(x, w, state=st, offsets=off)
    dx, _, _, dst = B.sla_conv_backward(x, w, x, state=st, grad_last=st, offsets=off)
    torch.cuda.synchronize()
    assert y.shape == dx.shape == (steps, d) and last.shape == dst.shape == st.shape
    assert (big == 7).all()

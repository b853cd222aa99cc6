"""Recurrences whose products of coefficients leave the range of their type, and
values that are not finite, across chunks and in both directions: element by
element against the formulas taken step by step in 64 bits."""
import numpy as np
import pytest
import torch

from preconditioned_cg_solver_amd import binding as B
from gpu_util import DEV, say
from test_gpu_linrec import check, make, reference, run
import seq_util as S

pytestmark = pytest.mark.gpu

# one step; up to 32 steps, which have a kernel of their own; either side of a
# chunk of 128 or 256 steps; several chunks; more than one look takes in
LENGTHS = [1, 31, 33, 127, 129, 255, 257, 300, 1100, 9000]


def stepwise(x, g, h0, mode, dh, dl):
    """The formulas step by step (dense)."""
    n, steps, d = x.shape
    with np.errstate(all="ignore"):
        a, b, keep = S.coefficients(x, g, mode)
        h, before = np.zeros_like(x), np.zeros_like(x)
        st = np.zeros((n, d)) if h0 is None else h0.copy()
        for t in range(steps):
            before[:, t] = st
            st = a[:, t] * st + b[:, t]
            h[:, t] = st
        dx, dg = np.zeros_like(x), np.zeros_like(x)
        mu = dl.copy()
        for t in range(steps - 1, -1, -1):
            lam = dh[:, t] + mu
            mu = a[:, t] * lam
            dx[:, t] = lam * keep[:, t]
            dg[:, t] = mu * (before[:, t] - x[:, t]) * keep[:, t] if mode == "sigmoid" else \
                lam * before[:, t]
    out = {"h": h, "last": st, "dx": dx, "dgate": dg}
    if mode == "sigmoid":
        # an infinite gradient times a difference that is zero in 32 bits, where
        # the state is known to some 100 roundings (of 2^-24): anything
        diff = np.abs(before - x) <= 2.0 ** -17 * (np.abs(before) + np.abs(x))
        out["dgate"][diff & np.isinf(dx)] = np.inf
        out["any"] = diff & np.isinf(dx)
    return out if h0 is None else dict(out, dh0=mu)


def check_kinds(got, want, clean, what):
    """NaN and infinities where the formulas have them; the rest as in the
    sequence without any, within its bounds."""
    want = dict(want)
    free = want.pop("any", None)
    for name, v in want.items():
        t = got[name].double().cpu().numpy()
        if name == "dgate" and free is not None:
            t = np.where(free, v, t)
        assert np.array_equal(np.isnan(t), np.isnan(v)), (what, name, "NaN")
        inf = np.isinf(v)
        assert np.array_equal(t[inf], v[inf]) and not np.any(np.isinf(t[~inf])), (what, name)
        ok = np.isfinite(v)
        ref, bound = clean[name]
        assert np.all(np.abs(t - ref)[ok] <= bound[ok]), (what, name, "error over bound")


@pytest.mark.parametrize("dt", ["f64", "f32", "bf16", "f16"])
@pytest.mark.parametrize("steps", LENGTHS)
def test_growth_from_a_zero_state(dt, steps):
    """Coefficients of 1.5 throughout: x is zero but for the last steps (padding
    in front), the gradient but for the first (no loss on the tail)."""
    say("recurrence growth from zero", dt, steps)
    n, d = 2, 70
    x, g, h0, dh, dl = make(dt, "linear", (n, steps), d, n, 30, h0=False)
    g[:] = 1.5
    x[:, :-5], dh[:, 5:], dl[:] = 0.0, 0.0, 0.0
    got = run(dt, "linear", x, g, None, None, dh, dl)
    check(got, reference(dt, "linear", x, g, None, None, dh, dl), (dt, steps))


@pytest.mark.parametrize("dt", ["f64", "f32", "bf16"])
def test_growth_from_a_zero_state_packed(dt):
    lens = [300, 0, 33, 1, 700, 129, 256]
    off = np.concatenate([[0], np.cumsum(lens)])
    say("recurrence growth from zero, packed", dt)
    x, g, h0, dh, dl = make(dt, "linear", (int(off[-1]),), 40, len(lens), 31, h0=False)
    g[:] = -1.75
    for a, b in zip(off[:-1], off[1:]):
        x[a:max(a, b - 3)], dh[min(b, a + 3):b] = 0.0, 0.0
    dl[:] = 0.0
    got = run(dt, "linear", x, g, None, off, dh, dl)
    check(got, reference(dt, "linear", x, g, None, off, dh, dl), dt)


@pytest.mark.parametrize("dt", ["f64", "f32", "bf16"])
@pytest.mark.parametrize("steps", [20, 64, 200, 300, 1100])
def test_large_coefficients_before_a_zero(dt, steps):
    """Two very large coefficients and a zero, and mirrored in time for the
    gradients, while the state and its gradient are zero."""
    say("recurrence large before zero", dt, steps)
    n, d = 2, 9
    big = {"f64": 1e200, "f32": 1e20, "bf16": 2.0 ** 66}[dt]
    x, g, h0, dh, dl = make(dt, "linear", (n, steps), d, n, 32, h0=False)
    g[:], x[:], dh[:], dl[:] = 0.5, 0.0, 0.0, 0.0
    for at in (0, steps // 2, steps - 6):
        g[:, at:at + 6] = np.array([big, big, 0.0, 0.0, big, big])[:, None]
    x[:, -1], dh[:, 0] = 1.0, 1.0
    got = run(dt, "linear", x, g, None, None, dh, dl)
    check(got, reference(dt, "linear", x, g, None, None, dh, dl), (dt, steps))


@pytest.mark.parametrize("dt", ["f64", "f32", "bf16"])
@pytest.mark.parametrize("first", [1, -1])
@pytest.mark.parametrize("steps", [40, 130, 300, 1100])
@pytest.mark.parametrize("turn", [2, 10, 20, 100])
def test_growth_and_decay_in_turn(dt, first, steps, turn):
    """Runs of `turn` steps that multiply the state by a large power of two, then
    as many that take it back: from one end of the type's range to the other."""
    say("recurrence growth and decay", dt, first, steps, turn)
    n, d = 1, 66
    x, g, h0, dh, dl = make(dt, "linear", (n, steps), d, n, 33)
    power = (1800 if dt == "f64" else 200) // turn
    e = np.where(np.arange(steps) // turn % 2 == 0, power, -power) * first
    ahead, behind = np.cumsum(e), np.cumsum(e[::-1])
    g[:] = (2.0 ** e)[:, None]
    x[:], dh[:] = 0.0, 0.0
    h0[:] = 2.0 ** -((ahead.max() + ahead.min()) // 2)
    dl[:] = 2.0 ** -((behind.max() + behind.min()) // 2)
    got = run(dt, "linear", x, g, h0, None, dh, dl)
    check(got, reference(dt, "linear", x, g, h0, None, dh, dl), (dt, first, steps, turn))


@pytest.mark.parametrize("dt", ["f64", "f32", "bf16"])
@pytest.mark.parametrize("n,steps,d", [(2, 33, 40), (2, 300, 70), (1, 3000, 64), (1, 300, 8200)])
def test_coefficients_on_both_sides_of_one(dt, n, steps, d):
    """Normal coefficients: a third of them grow the state, which stays bounded."""
    say("recurrence normal coefficients", dt, n, steps, d)
    x, g, h0, dh, dl = make(dt, "linear", (n, steps), d, n, 34)
    g = torch.from_numpy(np.random.default_rng(35).standard_normal(g.shape)).to(
        {"f64": torch.float64, "f32": torch.float32, "bf16": torch.bfloat16}[dt]).double().numpy()
    got = run(dt, "linear", x, g, h0, None, dh, dl)
    check(got, reference(dt, "linear", x, g, h0, None, dh, dl), (dt, n, steps, d))


@pytest.mark.parametrize("mode", ["linear", "sigmoid"])
@pytest.mark.parametrize("dt", ["f64", "f32", "bf16", "f16"])
@pytest.mark.parametrize("steps", [20, 200, 300, 1100, 9000])
@pytest.mark.parametrize("strength", ["weak", "strong"])
def test_infinite_states_stay_infinite(mode, dt, steps, strength):
    """An infinite state, or gradient, that shrinks at every step stays infinite
    however small the product of the coefficients gets."""
    say("recurrence infinite states", mode, dt, steps, strength)
    n, d = 2, 67
    x, g, h0, dh, dl = make(dt, mode, (n, steps), d, n, 36)
    # channels 40 on: coefficients of a quarter (negative ones: the sign turns),
    # or small enough for a few steps to underflow
    small = {"linear": {"weak": -0.25, "strong": 2.0 ** -14}, "sigmoid": {"weak": -1.0,
             "strong": -40.0 if dt != "f64" else -300.0}}[mode][strength]
    g[:, :, 40:] = small
    base = reference(dt, mode, x, g, h0, None, dh, dl)
    x, h0, dh, dl = (v.copy() for v in (x, h0, dh, dl))
    h0[0, 41], h0[1, 42] = np.inf, -np.inf
    x[0, steps // 3, 43], x[1, 2, 44] = -np.inf, np.inf
    dl[0, 45], dl[1, 46] = np.inf, -np.inf
    dh[0, steps // 2, 47], dh[1, steps - 2, 48] = np.inf, -np.inf
    h0[1, 50], x[0, 5, 51], dl[0, 52], dh[1, 7, 53] = (np.nan,) * 4
    want = stepwise(x, g, h0, mode, dh, dl)
    assert np.all(np.isinf(want["h"][0, :, 41])) and np.all(np.isinf(want["dx"][0, :, 45]))
    got = run(dt, mode, x, g, h0, None, dh, dl)
    check_kinds(got, want, base, (mode, dt, steps, strength))


@pytest.mark.parametrize("mode", ["linear", "sigmoid"])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,steps,d", [(2, 600, 68), (2, 600, 4100), (3, 100, 64)])
def test_infinite_states_in_packs_of_channels(mode, dt, n, steps, d):
    """The same where a thread has several channels, in narrow and wide chunks and
    in a single one; a coefficient of zero makes a NaN of an infinite state and
    forgets a finite one."""
    say("recurrence infinite states in packs", mode, dt, n, steps, d)
    x, g, h0, dh, dl = make(dt, mode, (n, steps), d, n, 40)
    cut = 0.0 if mode == "linear" else -np.inf
    g[:, :, 40:] = 2.0 ** -14 if mode == "linear" else -40.0
    g[:, 70, 51:56] = cut
    base = reference(dt, mode, x, g, h0, None, dh, dl)
    x, h0, dh, dl = (v.copy() for v in (x, h0, dh, dl))
    h0[0, 41], h0[1, 42], h0[0, 52] = np.inf, -np.inf, np.inf
    x[0, 33, 43], x[0, 20, 53] = -np.inf, np.inf
    dl[0, 45], dl[1, 54] = np.inf, -np.inf
    dh[0, steps // 2, 47], dh[1, 80, 55] = np.inf, np.inf
    want = stepwise(x, g, h0, mode, dh, dl)
    assert np.all(np.isnan(want["h"][0, 70:, 52:54])) and np.all(np.isinf(want["h"][0, :, 41]))
    assert np.all(np.isnan(want["dx"][1, :70, 54:56]))
    got = run(dt, mode, x, g, h0, None, dh, dl)
    check_kinds(got, want, base, (mode, dt, n, steps, d))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_zero_coefficient_and_an_infinite_state(dt):
    """What the formulas make of it: not a number, from there on."""
    say("recurrence zero times infinity", dt)
    n, steps, d = 1, 700, 6
    x, g, h0, dh, dl = make(dt, "linear", (n, steps), d, n, 37)
    base = reference(dt, "linear", x, g, h0, None, dh, dl)
    x, g = x.copy(), g.copy()
    h0[0, 1], x[0, 150, 2] = np.inf, -np.inf
    g[0, 400, 1:3] = 0.0
    want = stepwise(x, g, h0, "linear", dh, dl)
    assert np.all(np.isnan(want["h"][0, 400:, 1:3])) and np.all(np.isinf(want["h"][0, 150:400, 2]))
    got = run(dt, "linear", x, g, h0, None, dh, dl)
    for k in ("h", "last"):
        check_kinds({k: got[k]}, {k: want[k]}, base, (dt, k))


@pytest.mark.parametrize("mode", ["linear", "sigmoid"])
def test_non_finite_values_packed(mode):
    """They stay in their own sequence and channel."""
    say("recurrence non-finite, packed", mode)
    lens = [400, 1, 0, 300, 700]
    off = np.concatenate([[0], np.cumsum(lens)])
    x, g, h0, dh, dl = make("f32", mode, (int(off[-1]),), 33, len(lens), 38)
    base = reference("f32", mode, x, g, h0, off, dh, dl)
    x, dh, h0 = x.copy(), dh.copy(), h0.copy()
    x[450, 3], x[700, 4], h0[4, 5], dh[300, 6], dh[1200, 7] = (
        np.inf, np.nan, -np.inf, np.inf, np.nan)
    got = run("f32", mode, x, g, h0, off, dh, dl)
    for s, (a, b) in enumerate(zip(off[:-1], off[1:])):
        cut = [v[None, a:b] for v in (x, g, dh)]
        want = stepwise(cut[0], cut[1], h0[s:s + 1], mode, cut[2], dl[s:s + 1])
        part = {k: (t[s:s + 1] if k in ("last", "dh0") else t[None, a:b]) for k, t in got.items()}
        clean = {k: tuple(v[s:s + 1] if k in ("last", "dh0") else v[None, a:b] for v in base[k])
                 for k in base}
        check_kinds(part, want, clean, (mode, s))


def test_same_bits_whichever_way_what_enters_was_found():
    """Chunks with and without maps of their own side by side."""
    say("recurrence determinism, chunks without maps")
    n, steps, d = 2, 5000, 130
    x, g, h0, dh, dl = make("f32", "linear", (n, steps), d, n, 39)
    g[:, 1000:1300, 5], x[:, :1299, 5], dh[:, 1001:, 5], dl[:, 5] = 3.0, 0.0, 0.0, 0.0
    h0[:, 5] = 0.0
    x[0, 2000, 70], dh[1, 3000, 71] = np.inf, np.nan
    first = run("f32", "linear", x, g, h0, None, dh, dl)
    for _ in range(5):
        again = run("f32", "linear", x, g, h0, None, dh, dl)
        for k in first:
            assert torch.equal(first[k].nan_to_num(7.0), again[k].nan_to_num(7.0)), k


@pytest.mark.parametrize("mode", ["linear", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [8192, 8191])
@pytest.mark.parametrize("packed", [False, True])
def test_16_bit_rows_past_the_caches(mode, dtype, d, packed):
    """Calls of more than 256 MB of 16-bit rows read and write past the caches:
    a quarter of the channels alone, which goes through them, has the same bits,
    in whole chunks and in the last ones of sequences, in packs of channels and one
    by one."""
    say("recurrence past the caches", mode, dtype, d, packed)
    n, steps = 4, 2000 + 77
    gen = torch.Generator(device=DEV).manual_seed(6)
    shape = (n * steps, d) if packed else (n, steps, d)
    x, g, dh = (torch.randn(shape, device=DEV, generator=gen).mul_(0.4).to(dtype)
                for _ in range(3))
    h0, dl = (torch.randn(n, d, device=DEV, generator=gen) for _ in range(2))
    off = torch.tensor([0, 1, 900, 900, n * steps], device=DEV) if packed else None

    def call(at):
        a, b, c = (t[..., at].contiguous() for t in (x, g, dh))
        s, e = h0[:, at].contiguous(), dl[:, at].contiguous()
        h, last, saved = B.sla_linrec_forward(a, b, h0=s, offsets=off, mode=mode, save=True)
        return [h, last, *B.sla_linrec_backward(a, b, saved, c, grad_last=e, h0=s, offsets=off,
                                                mode=mode)]

    part = slice(4096, 6144 + d % 2)  # as many channels a thread
    for a, b in zip(call(slice(0, d)), call(part)):
        assert torch.equal(a[..., part], b)


def test_sizes_are_those_of_a_call():
    say("recurrence sizes")
    x = torch.randn(2, 700, 96, device=DEV)
    _, _, saved = B.sla_linrec_forward(x, x, save=True)
    assert B.sla_linrec_sizes(x, x)[0] == saved.numel() * 4
    off = torch.tensor([0, 700, 1400], device=DEV)
    flat = x.view(1400, 96)
    _, _, saved = B.sla_linrec_forward(flat, flat, offsets=off, save=True)
    assert B.sla_linrec_sizes(flat, flat, off)[0] == saved.numel() * 4

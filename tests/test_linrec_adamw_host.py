"""The recurrences and the AdamW step without a GPU: what the C entry points and
the binding refuse, their sizes, and the references that the GPU tests use."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from preconditioned_cg_solver_amd import binding as B
import seq_util as S

OK, INVALID, UNSUPPORTED = 0, -1, -2


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        from preconditioned_cg_solver_amd import build
        build.build()
    return B.lib()


def shape(**kw):
    q = dict(n_seq=2, steps=600, dim=96, d_offsets=None, dtype=B.SLA_BF16,
             gate=B.SLA_GATE_SIGMOID)
    q.update(kw)
    return B.LinrecShape(**q)


def sizes(L, q):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    st = L.sla_linrec_sizes(ctypes.byref(q), ctypes.byref(a), ctypes.byref(b))
    return st, a.value, b.value


@pytest.mark.parametrize("kw,want", [
    (dict(n_seq=-1), INVALID), (dict(steps=-1), INVALID), (dict(dim=-1), INVALID),
    (dict(dtype=9), INVALID), (dict(gate=2), INVALID), (dict(steps=1 << 41), UNSUPPORTED),
    (dict(dim=1 << 28), UNSUPPORTED), (dict(n_seq=(1 << 31) - 1, dim=1 << 20), UNSUPPORTED),
    (dict(n_seq=1 << 20, steps=1 << 30), UNSUPPORTED)])
def test_shapes_refused(L, kw, want):
    assert sizes(L, shape(**kw))[0] == want
    assert L.sla_last_error()


def test_sizes(L):
    assert sizes(L, shape(n_seq=0)) == (OK, 0, 0)
    assert sizes(L, shape(steps=0)) == (OK, 0, 0)
    assert sizes(L, shape(steps=1))[2] == 0  # a serving step needs no workspace
    st, saved, work = sizes(L, shape())
    assert st == OK and saved > 0 and work > saved
    # states are fp32 for 16-bit sequences, fp64 for fp64
    assert sizes(L, shape(dtype=B.SLA_F64))[1] >= 2 * saved
    assert L.sla_linrec_sizes(None, None, None) == INVALID
    assert L.sla_linrec_sizes(ctypes.byref(shape()), None, None) == INVALID


P = [ctypes.c_void_p(0x1000 * (k + 1)) for k in range(12)]  # never dereferenced


def forward(L, q, x=P[0], xs=1, xt=1, g=P[1], h0=P[2], h=P[3], last=P[4], saved=None, work=P[6],
            nw=1 << 40):
    return L.sla_linrec_forward(ctypes.byref(q) if q else None, x, xs, xt, g, 1, 1, h0, h, last,
                                saved, work, nw, None)


def backward(L, q, x=P[0], g=P[1], saved=P[2], d=P[3], dt=1, dx=P[4], dg=P[5], work=P[6],
             nw=1 << 40):
    return L.sla_linrec_backward(ctypes.byref(q) if q else None, x, 1, 1, g, 1, 1, None, saved, d,
                                 1, dt, None, dx, dg, None, work, nw, None)


def test_linrec_arguments_refused(L):
    q = shape()
    for bad in (dict(x=None), dict(g=None), dict(h=None), dict(xs=-1), dict(xt=-5),
                dict(h=P[0]), dict(h=P[1]), dict(work=None), dict(nw=8),
                dict(work=ctypes.c_void_p(0x1008))):
        assert forward(L, q, **bad) == INVALID, bad
        assert L.sla_last_error()
    assert forward(L, None) == INVALID
    for bad in (dict(x=None), dict(g=None), dict(saved=None), dict(dx=None), dict(dg=None),
                dict(dt=-1), dict(dx=P[0]), dict(dg=P[3]), dict(dx=P[2]), dict(dg=P[4]),
                dict(work=None), dict(nw=8)):
        assert backward(L, q, **bad) == INVALID, bad
    assert backward(L, None) == INVALID
    # nothing to do: no argument is looked at
    assert forward(L, shape(n_seq=0), x=None, g=None, h=None, work=None, nw=0) == OK
    assert backward(L, shape(dim=0), x=None, g=None, saved=None, dx=None, dg=None, work=None,
                    nw=0) == OK


def test_any_offsets_stay_within_the_rows():
    """The arithmetic that places a packed sequence's chunks, for offsets that
    ascend and for arbitrary ones: a chunk's row and those that it looks at
    (`after` following ones) are rows of the call, its steps steps of it."""
    rng = np.random.default_rng(3)
    for case in range(400):
        n, steps = int(rng.integers(1, 9)), int(rng.integers(0, 2000))
        chunk = int(rng.choice([32, 64, 128, 256, 512]))
        rows = steps // chunk + n
        off = rng.integers(-5000, 5000, n + 1) if case % 2 else \
            np.sort(rng.integers(0, steps + 1, n + 1))
        if not case % 2:
            off[0], off[-1] = 0, steps
        first = [min(max(int(o), 0), steps) // chunk + s for s, o in enumerate(off[:-1])]
        covered = np.zeros(steps, int)
        for row in range(rows):
            lo, hi = 0, n
            while hi - lo > 1:
                mid = (lo + hi) >> 1
                lo, hi = (mid, hi) if first[mid] <= row else (lo, mid)
            o0 = min(max(int(off[lo]), 0), steps)
            o1 = min(max(int(off[lo + 1]), o0), steps)
            c = max(row - (o0 // chunk + lo), 0)
            after = max(-(-(o1 - o0) // chunk) - 1 - c, 0)
            assert c <= row and row + after <= rows - 1
            a, b = o0 + c * chunk, min(o0 + (c + 1) * chunk, o1)
            if a < b:
                assert 0 <= a and b <= steps
                covered[a:b] += 1
        if not case % 2:
            assert np.all(covered == 1)


# ----- AdamW -----

def tensor(p=0x10000, n=1000, dt=B.SLA_F32, gd=None, copy=None):
    return B.AdamwTensor(p, copy, n, dt, dt if gd is None else gd)


def adam_sizes(L, ts, bits=32, n=None):
    arr = (B.AdamwTensor * max(len(ts), 1))(*ts)
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_int64()
    st = L.sla_adamw_sizes(arr, len(ts) if n is None else n, bits, ctypes.byref(a),
                           ctypes.byref(b), ctypes.byref(c))
    return st, a.value, b.value, c.value


@pytest.mark.parametrize("t,want", [
    (tensor(dt=7), INVALID), (tensor(gd=7), INVALID), (tensor(n=-1), INVALID),
    (tensor(p=None), INVALID), (tensor(p=0x10002), INVALID),
    (tensor(copy=0x20001), INVALID), (tensor(dt=B.SLA_F16), UNSUPPORTED),
    (tensor(dt=B.SLA_BF16, gd=B.SLA_F32), UNSUPPORTED),
    (tensor(dt=B.SLA_F64, gd=B.SLA_F32), UNSUPPORTED),
    (tensor(dt=B.SLA_BF16, copy=0x20000), UNSUPPORTED)])
def test_adamw_tensors_refused(L, t, want):
    assert adam_sizes(L, [t])[0] == want
    assert L.sla_last_error()


def test_adamw_sizes(L):
    ts = [tensor(n=n) for n in (0, 1, 256, 257)]
    st, state, table, padded = adam_sizes(L, ts)
    assert st == OK and padded == 256 * 4 and state == 8 * padded and table > 0
    assert adam_sizes(L, ts, 8)[1] == 2 * padded + 4 * 4
    assert adam_sizes(L, ts, 16)[0] == UNSUPPORTED
    assert adam_sizes(L, [], 8) == (OK, 0, 0, 0)
    assert adam_sizes(L, ts, n=-1)[0] == INVALID


def test_adamw_calls_refused(L):
    h, arr = ctypes.c_void_p(), (B.AdamwTensor * 1)(tensor())
    create = L.sla_adamw_create
    big = 1 << 30
    assert create(None, arr, 1, 32, P[0], big, P[1], big, None) == INVALID
    assert create(ctypes.byref(h), None, 1, 32, P[0], big, P[1], big, None) == INVALID
    assert create(ctypes.byref(h), arr, 1, 32, None, big, P[1], big, None) == INVALID
    assert create(ctypes.byref(h), arr, 1, 32, P[0], 10, P[1], big, None) == INVALID
    assert create(ctypes.byref(h), arr, 1, 32, P[0], big, P[1], 10, None) == INVALID
    assert create(ctypes.byref(h), arr, 1, 32, ctypes.c_void_p(0x1010), big, P[1], big,
                  None) == INVALID
    assert create(ctypes.byref(h), arr, 1, 5, P[0], big, P[1], big, None) == UNSUPPORTED
    assert not h
    hyper = B.AdamwHyper(1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 0)
    assert L.sla_adamw_step(None, None, ctypes.byref(hyper), None, None) == INVALID
    assert L.sla_adamw_get_state(None, P[0], P[1], None) == INVALID
    assert L.sla_adamw_set_state(None, P[0], P[1], None) == INVALID
    assert L.sla_adamw_destroy(None) == OK


# ----- the binding -----

class FakeCuda:
    """Shape, dtype, strides and device of a tensor on the GPU."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.float32, stride=None, device="cuda:0"):
        self.shape, self.dtype, self.device = tuple(shape), dtype, torch.device(device)
        st, s = [], 1
        for k in reversed(self.shape):
            st.insert(0, s)
            s *= k
        self._stride = tuple(stride) if stride else tuple(st)
        self._contig = stride is None

    def stride(self, *a):
        return self._stride

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return self._contig

    def data_ptr(self):
        return 0x10000

    def detach(self):
        return self


X = FakeCuda((2, 10, 8))


@pytest.mark.parametrize("kw", [
    dict(x=FakeCuda((2, 10))), dict(x=FakeCuda((2, 10, 8), torch.int32)),
    dict(gate=FakeCuda((2, 10, 7))), dict(gate=FakeCuda((2, 10, 8), torch.bfloat16)),
    dict(gate=FakeCuda((2, 10, 8), stride=(160, 16, 2))), dict(mode="tanh"),
    dict(h0=FakeCuda((2, 7))), dict(h0=FakeCuda((2, 8), torch.float64)),
    dict(h0=FakeCuda((2, 8), device="cuda:1")), dict(gate=torch.zeros(2, 10, 8)),
    dict(offsets=FakeCuda((3,), torch.int64)),
    dict(x=FakeCuda((10, 8)), gate=FakeCuda((10, 8)), offsets=FakeCuda((3,), torch.int32)),
    dict(h_last=FakeCuda((3, 8)))])
def test_binding_refuses_sequences(kw):
    args = dict(x=X, gate=X)
    args.update(kw)
    with pytest.raises(ValueError):
        B.sla_linrec_forward(args.pop("x"), args.pop("gate"), **args)


def test_binding_refuses_gradients(L):
    with pytest.raises(ValueError):
        B.sla_linrec_backward(X, X, FakeCuda((3,)), FakeCuda((2, 10, 7)))
    with pytest.raises(ValueError):  # saved of another size
        B.sla_linrec_backward(X, X, FakeCuda((3,)), X)


def test_binding_refuses_parameters(L):
    with pytest.raises(ValueError):
        B.sla_adamw_create([FakeCuda((4, 4), stride=(8, 2))])
    with pytest.raises(ValueError):
        B.sla_adamw_create([FakeCuda((4,), torch.int64)])
    with pytest.raises(ValueError):
        B.sla_adamw_create([FakeCuda((4,))], copies=[FakeCuda((4,))])
    with pytest.raises(ValueError):
        B.sla_adamw_create([FakeCuda((4,))], grad_dtype=[torch.float32, torch.float32])
    with pytest.raises(ValueError):
        B.sla_adamw_create([FakeCuda((4,)), FakeCuda((4,), device="cuda:1")])
    with pytest.raises(B.SlaError):
        B.sla_adamw_create([FakeCuda((4,), torch.bfloat16)], grad_dtype=torch.float32)


# ----- the references themselves -----

@pytest.mark.parametrize("mode", ["linear", "sigmoid"])
@pytest.mark.parametrize("offsets", [None, [0, 3, 3, 9]])
def test_reference_gradients_against_differences(mode, offsets):
    r = np.random.default_rng(1)
    lead, n, d = ((2, 5), 2, 3) if offsets is None else ((9,), 3, 3)
    x, g = r.standard_normal((*lead, d)), 0.5 * r.standard_normal((*lead, d))
    h0, dh, dl = (r.standard_normal(s) for s in ((n, d), (*lead, d), (n, d)))

    def loss(x, g, h0):
        o = S.recurrence(x, g, h0, offsets, mode)
        return (o["h"][0] * dh).sum() + (o["last"][0] * dl).sum()

    want = S.recurrence(x, g, h0, offsets, mode, dh, dl)
    for k, name in enumerate(("dx", "dgate", "dh0")):
        args = [x, g, h0]
        for idx in np.ndindex(args[k].shape):
            e = np.zeros_like(args[k])
            e[idx] = 1e-6
            up, dn = list(args), list(args)
            up[k], dn[k] = args[k] + e, args[k] - e
            diff = (loss(*up) - loss(*dn)) / 2e-6
            assert abs(diff - want[name][0][idx]) <= 1e-7 * (1 + abs(diff)), (name, idx)


def test_random_bits_are_even():
    """Each of the 32 bits is set in half of the elements, and the bits used for
    m, v and a bf16 parameter do not follow each other: within 5 standard
    deviations of n / 2 coin flips."""
    n = 1 << 18
    a = S.noise(7, 11, n)
    b = S.mix(a + np.uint64(0x6A09E667))
    bound = 5 * math.sqrt(n) / 2
    bits = [((v >> np.uint64(k)) & np.uint64(1)).astype(bool) for v in (a, b) for k in range(32)]
    for k, v in enumerate(bits):
        assert abs(int(v.sum()) - n / 2) <= bound, k
        assert abs(int((v[1:] ^ v[:-1]).sum()) - n / 2) <= bound, k
    for k in range(16):
        assert abs(int((bits[k] ^ bits[16 + k]).sum()) - n / 2) <= bound
        assert abs(int((bits[k] ^ bits[32 + k]).sum()) - n / 2) <= bound
    c = S.noise(7, 12, n)
    assert abs(int(((a ^ c) & np.uint64(1)).sum()) - n / 2) <= bound


def test_levels_of_the_8_bit_form():
    x = np.zeros(256, np.float32)
    x[:6] = [1.0, 0.5, 2.0 ** -30, 2.0 ** -40, 1.0624, -0.3]
    none = np.zeros(256, np.uint64)
    v = S.levels(np.abs(x), none, 254, 1)
    assert v[0] == 1.0 and v[1] == 0.5 and v[2] == np.float32(2.0 ** -30)
    assert 0 < v[3] < 2.0 ** -31            # held at the lowest level
    assert v[4] == 1.0                       # dropped to three mantissa bits
    m = S.levels(x, none, 126, 0)
    assert m[2] == 0 and m[5] == np.float32(-0.28125)
    up = S.levels(np.abs(x), none + np.uint64(0xFFFFF), 254, 1)
    assert up[4] == 1.125 and up[0] == 1.0

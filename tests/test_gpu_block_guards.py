"""What a sequence block's operators write lies within the arrays that they are given: every
output, the kept states and the workspaces stand between guards, called through the C ABI with
workspaces of the size that was asked for."""
import ctypes

import pytest
import torch

from preconditioned_cg_solver_amd import binding as B
from block_gpu import DT, make, own_of
from gpu_util import say

pytestmark = pytest.mark.gpu
GUARD, MARK = 8192, 0xA5
ASCENDING = [5, 5, 21, 22, 60, 60]             # rows of no sequence at both ends
ARBITRARY = [40, -3, 900, 12, 12, -70]
FAR = [-(1 << 63), (1 << 63) - 1, 7, 1 << 40, -(1 << 40), 31]


class Arena:
    """Arrays in one buffer, bytes that nobody may write around each."""

    def __init__(self, nbytes=1 << 26):
        self.all = torch.full((nbytes,), MARK, dtype=torch.uint8, device="cuda")
        self.free, self.at = torch.ones(nbytes, dtype=torch.bool, device="cuda"), GUARD

    def __call__(self, shape, dtype):
        n = int(torch.Size(shape).numel()) * dtype.itemsize
        view = self.all[self.at:self.at + n]
        self.free[self.at:self.at + n] = False
        self.at += -(-n // 256) * 256 + GUARD
        assert self.at <= self.all.numel()
        view.fill_(0xFF)  # NaN
        return view.view(dtype).view(shape)

    def work(self, n):
        return self((n,), torch.uint8)

    def check(self):
        torch.cuda.synchronize()
        assert ((self.all == MARK) | ~self.free).all()


def at(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def marks(off, steps):
    return None if off is None else torch.tensor(off, device="cuda")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [3, 256, 260])
@pytest.mark.parametrize("off", [None, ASCENDING, ARBITRARY, FAR])
@pytest.mark.parametrize("steps", [7, 70, 300])
def test_conv(dtype, d, off, steps):
    say("conv between guards", dtype, d, off, steps)
    r, room, o = make(0, dtype), Arena(), marks(off, steps)
    n = 2 if off is None else len(off) - 1
    lead = (n, steps) if off is None else (steps,)
    x, dy, w, b = r(*lead, d), r(*lead, d), r.own(d, 4), r.own(d)
    st, dl = r(n, 3, d), r(n, 3, d)
    T, C = DT[dtype], own_of(dtype)
    y, last, dx = room((*lead, d), T), room((n, 3, d), T), room((*lead, d), T)
    dw, db, dst = room((d, 4), C), room((d,), C), room((n, 3, d), T)
    q = B.ConvShape(n, steps, d, 4, at(o), B._DTYPES[T], B.SLA_ACT_SILU)
    size = B._conv_sizes(q)
    work, L = room.work(size), B.lib()
    if off is not None:
        B._check(L.sla_rows_clear(at(o), n, steps, d, q.dtype, at(y), stream()))
    B._check(L.sla_conv_forward(ctypes.byref(q), at(x), steps * d, d, at(w), at(b), at(st), at(y),
                                at(last), stream()))
    B._check(L.sla_conv_backward(ctypes.byref(q), at(x), steps * d, d, at(w), at(b), at(st), at(dy),
                                 steps * d, d, at(dl), at(dx), at(dw), at(db), at(dst), at(work),
                                 size, stream()))
    room.check()
    if off in (None, ASCENDING) and (off is None or steps >= off[-1]):
        y1, last1 = B.sla_conv_forward(x, w, bias=b, state=st, offsets=o)
        g = B.sla_conv_backward(x, w, dy, bias=b, state=st, grad_last=dl, offsets=o)
        for p, s in zip((y, last, dx, dw, db, dst), (y1, last1, *g)):
            assert torch.equal(p, s)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("d,N,groups", [(20, 16, 1), (23, 3, 1), (24, 8, 3), (130, 16, 1)])
@pytest.mark.parametrize("off", [None, ASCENDING, ARBITRARY, FAR])
@pytest.mark.parametrize("steps", [7, 70, 300])
def test_scan(dtype, d, N, groups, off, steps):
    say("scan between guards", dtype, d, N, groups, off, steps)
    r, room, o = make(1, dtype), Arena(), marks(off, steps)
    n = 2 if off is None else len(off) - 1
    lead = (n, steps) if off is None else (steps,)
    T, C = DT[dtype], own_of(dtype)
    x, dt, z, dy = (r(*lead, d) for _ in range(4))
    bs, cs = r(*lead, groups, N), r(*lead, groups, N)
    A, D, bias, h0, dl = -r.own(d, N).abs(), r.own(d), r.own(d) - 2, r.own(n, d, N), r.own(n, d, N)
    q = B.SelscanShape(n, steps, d, N, groups, at(o), B._DTYPES[T], 1)
    sizes = [ctypes.c_size_t() for _ in range(3)]
    L = B.lib()
    B._check(L.sla_selscan_sizes(ctypes.byref(q), *(ctypes.byref(s) for s in sizes)))
    n_saved, n_fwd, n_back = (s.value for s in sizes)
    rows, shared = (steps * d, d), (steps * groups * N, groups * N)
    given = B.SelscanIn(at(x), at(dt), at(z), at(bs), at(cs), *rows, *rows, *rows, *shared, *shared,
                        at(A), at(D), at(bias), at(h0))
    y, last, saved = room((*lead, d), T), room((n, d, N), C), room.work(n_saved)
    fwd, back = room.work(n_fwd), room.work(n_back)
    if off is not None:
        B._check(L.sla_rows_clear(at(o), n, steps, d, q.dtype, at(y), stream()))
    B._check(L.sla_selscan_forward(ctypes.byref(q), ctypes.byref(given), at(y), at(last), at(saved),
                                   at(fwd) if n_fwd else None, n_fwd, stream()))
    out = [room(s, t) for s, t in (((*lead, d), T), ((*lead, d), T), ((*lead, d), T),
                                   ((*lead, groups, N), T), ((*lead, groups, N), T), ((d, N), C),
                                   ((d,), C), ((d,), C), ((n, d, N), C))]
    grads = B.SelscanGrads(*(at(t) for t in out))
    B._check(L.sla_selscan_backward(ctypes.byref(q), ctypes.byref(given), at(saved), at(dy), *rows,
                                    at(dl), ctypes.byref(grads), at(back), n_back, stream()))
    few, after = room((*lead, d), T), room((n, d, N), C)  # without kept states
    B._check(L.sla_selscan_forward(ctypes.byref(q), ctypes.byref(given), at(few), at(after), None,
                                   at(fwd) if n_fwd else None, n_fwd, stream()))
    room.check()
    if off in (None, ASCENDING) and (off is None or steps >= off[-1]):
        kw = dict(D=D, z=z, dt_bias=bias, h0=h0, offsets=o)
        y1, last1, s1 = B.sla_selscan_forward(x, dt, A, bs, cs, **kw, save=True)
        dx, ddt, dA, dB, dC, dD, dz, dbias, dh0 = B.sla_selscan_backward(x, dt, A, bs, cs, s1, dy,
                                                                         grad_last=dl, **kw)
        for p, s in zip((y, last, *out), (y1, last1, dx, ddt, dz, dB, dC, dA, dD, dbias, dh0)):
            assert torch.equal(p, s)


# a way to take a row each: see the norms' own tests
@pytest.mark.parametrize("dtype,dim", [("bf16", 8), ("bf16", 33), ("bf16", 512), ("bf16", 2048),
                                       ("bf16", 4097), ("bf16", 8192), ("bf16", 16384),
                                       ("bf16", 16400), ("f32", 1000), ("f32", 1023), ("f32", 8196),
                                       ("f64", 4098)])
@pytest.mark.parametrize("rows", [1, 3, 1100])
def test_norms(dtype, dim, rows):
    if rows * dim > 1 << 23:
        rows = 530  # more rows than teams of 16 waves
    say("norms between guards", dtype, dim, rows)
    r, room = make(2, dtype), Arena(1 << 28)
    T, C = DT[dtype], own_of(dtype)
    x, g, res, do = (r(rows, dim) for _ in range(4))
    w, sc = r.own(dim), r.own(dim)
    q = B.NormShape(rows, dim, B._DTYPES[T], B._DTYPES[T], 1e-5)
    n, L = B._norm_sizes(q), B.lib()
    y, s, rstd = room((rows, dim), T), room((rows, dim), T), room((rows,), C)
    work = room.work(n)
    B._check(L.sla_norm_in_forward(ctypes.byref(q), at(x), dim, at(res), dim, at(sc), at(w), at(y),
                                   at(s), at(rstd), stream()))
    dx, dres = room((rows, dim), T), room((rows, dim), T)
    dw, dsc = room((dim,), C), room((dim,), C)
    B._check(L.sla_norm_in_backward(ctypes.byref(q), at(do), at(g), at(x), dim, at(res), dim, at(sc),
                                    at(w), at(rstd), at(dx), at(dres), at(dw), at(dsc), at(work), n,
                                    stream()))
    room.check()
    got = [t.clone() for t in (y, s, rstd, dx, dres, dw, dsc)]
    want = B.sla_norm_in_forward(x, w, residual=res, scale=sc)
    want += B.sla_norm_in_backward(do, x, w, want[2], residual=res, scale=sc, grad_r=g)
    assert all(torch.equal(p, v) for p, v in zip(got[:5], want[:5]))
    assert torch.equal(got[5], want[5]) and torch.equal(got[6], want[6])
    B._check(L.sla_norm_out_forward(ctypes.byref(q), 0, at(x), dim, at(g), dim, at(res), dim, at(sc),
                                    at(w), at(y), at(rstd), stream()))
    B._check(L.sla_norm_out_backward(ctypes.byref(q), 0, at(do), at(x), dim, at(g), dim, at(sc),
                                     at(w), at(rstd), at(dx), at(dres), at(dw), at(dsc), at(work), n,
                                     stream()))
    room.check()
    out, rs = B.sla_norm_out_forward(x, w, gate=g, residual=res, scale=sc)
    back = B.sla_norm_out_backward(do, x, w, rs, gate=g, scale=sc)
    assert all(torch.equal(p, v) for p, v in zip((y, rstd, dx, dres, dw, dsc), (out, rs, *back)))

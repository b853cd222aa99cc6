"""Recurrences and AdamW steps that need more threads than one launch has
(2^32 - 1), and element places beyond 2^32."""
import numpy as np
import pytest
import torch

from preconditioned_cg_solver_amd import binding as B
from gpu_util import DEV, say
import seq_util as S

pytestmark = pytest.mark.gpu


def room(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB")


def test_recurrence_of_many_single_steps():
    """8.5 million sequences of one step: as many workgroups of 512 threads in
    the backward pass."""
    n = 8_500_000
    say("recurrence, many sequences of a step", n)
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, g, dh = (torch.randn(n, 1, 1, device=DEV, generator=gen) for _ in range(3))
    h0, dl = (torch.randn(n, 1, device=DEV, generator=gen) for _ in range(2))
    h, last, saved = B.sla_linrec_forward(x, g, h0=h0, mode="linear", save=True)
    dx, dg, dh0 = B.sla_linrec_backward(x, g, saved, dh, grad_last=dl, h0=h0, mode="linear")
    x, g, dh, h0, dl = (t.reshape(-1).double() for t in (x, g, dh, h0, dl))
    lam = dh + dl
    # three roundings of the terms at most
    for got, want, size in ((h, g * h0 + x, (g * h0).abs() + x.abs()),
                            (last, g * h0 + x, (g * h0).abs() + x.abs()),
                            (dx, lam, dh.abs() + dl.abs()),
                            (dg, lam * h0, (dh.abs() + dl.abs()) * h0.abs()),
                            (dh0, g * lam, g.abs() * (dh.abs() + dl.abs()))):
        off = (got.reshape(-1).double() - want).abs()
        assert bool((off <= 4 * S.U32 * size + 2.0 ** -140).all())


@pytest.mark.parametrize("packed", [False, True])
def test_recurrence_of_many_chunks(packed):
    """More chunks than a launch has workgroups, joined in twos and threes: the
    first and the last sequences have the bits of calls of their own."""
    room(60)
    n, steps = (2_900_000, 300) if not packed else (4_300_000, 140)
    say("recurrence, many chunks", n, steps, packed)
    gen = torch.Generator(device=DEV).manual_seed(2)

    def rows():
        return torch.empty(n, steps, 1, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)

    x, g, dh = rows(), rows(), rows()
    h0, dl = (torch.randn(n, 1, device=DEV, generator=gen) for _ in range(2))

    def call(at):
        a, b, c = (t[at].contiguous() for t in (x, g, dh))
        k, off = a.shape[0], None
        if packed:
            a, b, c = (t.view(k * steps, 1) for t in (a, b, c))
            off = torch.arange(k + 1, device=DEV) * steps
        h, last, saved = B.sla_linrec_forward(a, b, h0=h0[at], offsets=off, save=True)
        dx, dg, dh0 = B.sla_linrec_backward(a, b, saved, c, grad_last=dl[at], h0=h0[at],
                                            offsets=off)
        return [t.view(k, -1) for t in (h, dx, dg)] + [last, dh0]

    whole = call(slice(0, n))
    torch.cuda.synchronize()
    for at in (slice(0, 64), slice(n // 2, n // 2 + 64), slice(n - 64, n)):
        for a, b in zip(whole, call(at)):
            assert torch.equal(a[at], b)


def test_serving_step_of_more_channels_than_threads():
    """4.3e9 channels, one a thread (an odd number of them a sequence)."""
    room(60)
    n, d = 2_100_000, 2049
    say("recurrence, serving step", n * d)
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, g = (torch.randn(1, 1, d, device=DEV, generator=gen).bfloat16() for _ in range(2))
    h, last, _ = B.sla_linrec_forward(x.expand(n, 1, d), g.expand(n, 1, d))
    one, state, _ = B.sla_linrec_forward(x, g)
    for at in (slice(0, 3), slice(n - 3, n)):
        assert torch.equal(h[at], one.expand(3, 1, d)) and torch.equal(last[at], state.expand(3, d))


def test_adamw_of_more_blocks_than_threads():
    """17.5e9 bf16 parameters with 8-bit states, one gradient for all five
    tensors: the step and the reading of the states at the first elements, at the
    first of the second launch and at the last, bit for bit; the setting at all."""
    room(220)
    size, k = 3_500_000_007, 5
    say("adamw, elements", size * k)
    gen = torch.Generator(device=DEV).manual_seed(4)
    g = torch.empty(size, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    ps = [torch.ones(size, dtype=torch.bfloat16, device=DEV) for _ in range(k)]
    opt = B.sla_adamw_create(ps, state_bits=8)
    B.sla_adamw_step(opt, [g] * k, step=1, seed=6, lr=1e-2)
    m, v = B.sla_adamw_get_state(opt)
    torch.cuda.synchronize()
    second = (2 ** 24 - 1) * 1024  # elements of the first launch's chunks of four blocks
    for at in (0, second - 512, opt.starts[1] + 5120, opt.starts[4] + size // 256 * 256 - 512):
        t = max(i for i in range(k) if opt.starts[i] <= at)
        i = at - opt.starts[t]
        n = min(1024, size - i)
        gr = S.pad_to_blocks([g[i:i + n].float().cpu().numpy()])
        key = int(S.mix(6 ^ int(S.mix(int(S.mix(1))))))
        e = at + np.arange(len(gr), dtype=np.uint64)
        hi = e >> np.uint64(32)
        keys = np.where(hi > 0, np.uint64(key) ^ S.mix(hi), np.uint64(key))
        r = S.mix((e & np.uint64(0xFFFFFFFF)) * np.uint64(0x9E3779B1) + keys)
        wm, wv = S.moments32(np.zeros_like(gr), np.zeros_like(gr), gr, 0.9, 0.999)
        wm = S.levels(wm, ((r & np.uint64(0xFFFF)) << np.uint64(4)) + np.uint64(8), 126, 0)
        wv = S.levels(wv, ((r >> np.uint64(16)) << np.uint64(4)) + np.uint64(8), 254, 1)
        assert np.array_equal(m[at:at + n].float().cpu().numpy(), wm[:n]), at
        assert np.array_equal(v[at:at + n].float().cpu().numpy(), wv[:n]), at
        # the first step moves each parameter by lr against its gradient's sign
        # (and by lr wd = 1e-4), to a bf16 neighbour: 2^-7 either way
        p = ps[t][i:i + n].float().cpu().numpy()
        want = 1 - 1e-2 * np.sign(gr[:n]) - 1e-4
        assert np.all(np.abs(p - want) <= 2.0 ** -7), at
    del m, v, g
    # ones, in the highest codes of their blocks, throughout
    ones = torch.ones(opt.padded, device=DEV)
    B.sla_adamw_set_state(opt, ones, ones)
    n = opt.padded
    assert bool((opt.state[:n] == 126).all()) and bool((opt.state[n:2 * n] == 254).all())
    bases = opt.state[2 * n:].view(torch.int16)
    assert bool((bases[:n // 256] == 1016 - 126).all())
    assert bool((bases[n // 256:] == 1016 - 254).all())

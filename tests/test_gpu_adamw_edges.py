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


def test_tensors_that_share_memory():
    """Two entries with the same memory are not stepped at once, whether whole,
    in part or through a copy; one of them alone is, as are neighbours."""
    say("adamw shared memory")
    flat = torch.ones(4000, device=DEV)
    low = torch.zeros(4000, device=DEV, dtype=torch.bfloat16)
    g = torch.full((1000,), 0.5, device=DEV)

    def step(spans, grads, copies=None):
        opt = B.sla_adamw_create([flat[a:a + 1000] for a in spans],
                                 copies=None if copies is None else
                                 [None if c is None else low[c:c + 1000] for c in copies])
        B.sla_adamw_step(opt, [g if k else None for k in grads], step=1, lr=1e-3)

    for spans, grads, copies in (([0, 0], (1, 1), None), ([0, 2000, 999], (1, 1, 1), None),
                                 ([1500, 0, 3000, 2499], (1, 1, 0, 1), None),
                                 ([0, 1000], (1, 1), [0, 999]),
                                 ([0, 1000, 2000], (1, 0, 1), [500, None, 0])):
        before = flat.clone()
        with pytest.raises(B.SlaError, match="share memory"):
            step(spans, grads, copies)
        assert torch.equal(flat, before) and not bool(low.any())
    for spans, grads, copies in (([0, 0], (1, 0), None), ([0, 2000, 999], (0, 1, 1), None),
                                 ([500, 0, 1000], (0, 1, 1), None),
                                 ([3000, 0, 1000], (1, 1, 1), None),
                                 ([0, 1000], (1, 1), [1000, 0]), ([0, 1000], (1, 0), [0, 999])):
        before = flat.clone()
        step(spans, grads, copies)
        moved = torch.zeros_like(flat, dtype=torch.bool)
        for a, k in zip(spans, grads):
            moved[a:a + 1000] |= bool(k)
        assert torch.equal(flat != before, moved), (spans, grads)


def test_many_tensors_with_the_same_memory():
    """Three entries of one weight; each may be the one that is stepped."""
    say("adamw tied three times")
    w, g = torch.ones(300, device=DEV), torch.ones(300, device=DEV)
    opt = B.sla_adamw_create([w, torch.ones(5, device=DEV), w, w])
    for k in (0, 2, 3):
        grads = [None, torch.ones(5, device=DEV), None, None]
        grads[k] = g
        before = w.clone()
        B.sla_adamw_step(opt, grads, step=1, lr=1e-2)
        assert bool((w < before).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_between_forward_and_backward_is_noticed(bits):
    """What autograd has saved and a step has written since is an error in the
    backward pass; what the step left alone is not."""
    say("adamw and autograd", bits)
    w, u, x = (torch.rand(300, device=DEV, requires_grad=True) for _ in range(3))
    low = torch.zeros(300, device=DEV, dtype=torch.bfloat16)
    opt = B.sla_adamw_create([w, u], state_bits=bits, copies=[low, None])
    g = torch.ones(300, device=DEV)
    for used, grads, fails in ((w, [g, None], True), (w, [g, g], True), (w, [None, g], False),
                               (u, [g, None], False), (low, [g, None], True),
                               (low, [None, g], False)):
        loss = (x * used).sum()
        B.sla_adamw_step(opt, grads, step=1, lr=1e-3)
        if fails:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()
        else:
            loss.backward()
    m, _ = B.sla_adamw_get_state(opt)
    if bits == 32:  # the handle's own buffer
        for write in (lambda: B.sla_adamw_step(opt, [g, g], step=2, lr=1e-3),
                      lambda: B.sla_adamw_set_state(opt, torch.zeros_like(m), torch.zeros_like(m))):
            loss = (x * m[:300]).sum()
            write()
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()


def test_a_last_state_that_autograd_has_saved():
    say("recurrence and autograd: h_last given")
    x, g = (torch.randn(2, 5, 8, device=DEV) for _ in range(2))
    scale = torch.rand(2, 8, device=DEV, requires_grad=True)
    state = torch.rand(2, 8, device=DEV)
    loss = (scale * state).sum()
    B.sla_linrec_forward(x, g, h0=state, h_last=state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_in_inference_mode():
    """Tensors without versions are written all the same."""
    say("operators in inference mode")
    with torch.inference_mode():
        x, g = (torch.randn(2, 5, 8, device=DEV) for _ in range(2))
        state = torch.rand(2, 8, device=DEV)
        _, want, _ = B.sla_linrec_forward(x, g, h0=state)
        B.sla_linrec_forward(x, g, h0=state, h_last=state)
        assert torch.equal(state, want)
        p = torch.ones(300, device=DEV)
        opt = B.sla_adamw_create([p])
        B.sla_adamw_step(opt, [torch.ones(300, device=DEV)], step=1, lr=1e-2)
        assert bool((p < 1).all())


def busy(stream):
    """Work of some milliseconds on the stream."""
    with torch.cuda.stream(stream):
        big = torch.ones(1 << 27, device=DEV)
        for _ in range(30):
            big.mul_(1.0)


def test_inputs_freed_while_another_stream_reads_them():
    """Memory of inputs given up right after a call on another stream is not
    handed out again before that call has read it."""
    say("operators on another stream, inputs freed")
    gen = torch.Generator(device=DEV).manual_seed(1)
    shape = (4, 700, 64)
    base = [torch.randn(shape, device=DEV, generator=gen) for _ in range(3)]
    h0 = torch.randn(4, 64, device=DEV, generator=gen)
    off = torch.tensor([0, 700, 1400, 2100, 2800], device=DEV)
    flat = [t.view(2800, 64) for t in base]
    h, last, saved = B.sla_linrec_forward(flat[0], flat[1], h0=h0, offsets=off, save=True)
    want = [h, last, *B.sla_linrec_backward(flat[0], flat[1], saved, flat[2], grad_last=h0, h0=h0,
                                            offsets=off)]
    s = torch.cuda.Stream()
    for _ in range(3):
        x, g, d = (t.clone() for t in flat)
        state, offsets = h0.clone(), off.clone()
        torch.cuda.synchronize()
        busy(s)
        h, last, saved = B.sla_linrec_forward(x, g, h0=state, offsets=offsets, save=True, stream=s)
        got = [h, last, *B.sla_linrec_backward(x, g, saved, d, grad_last=state, h0=state,
                                               offsets=offsets, stream=s)]
        sizes = [(t.shape, t.dtype) for t in (x, g, d, state, offsets)]
        del x, g, d, state, offsets, saved
        for k in range(4):  # would take the same memory, if it were free
            for shp, dt in sizes:
                torch.full(shp, 77, dtype=dt, device=DEV)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("given", [True, False])
def test_handle_freed_while_another_stream_steps(given):
    """The same for an AdamW handle's memory, its parameters and gradients."""
    say("adamw on another stream, handle freed", given)
    n = 1 << 20
    p0, g0 = torch.randn(n, device=DEV), torch.randn(n, device=DEV)
    ref = p0.clone()
    o = B.sla_adamw_create([ref], state_bits=8)
    for t in (1, 2):
        B.sla_adamw_step(o, [g0], step=t, lr=1e-2)
    s = torch.cuda.Stream()
    for _ in range(3):
        p, g, scale = p0.clone(), g0.clone(), torch.ones(1, device=DEV)
        opt = B.sla_adamw_create([p], state_bits=8)
        torch.cuda.synchronize()
        busy(s)
        with torch.cuda.stream(s) if not given else torch.cuda.stream(torch.cuda.current_stream()):
            for t in (1, 2):
                B.sla_adamw_step(opt, [g], step=t, lr=1e-2, grad_scale=scale,
                                 stream=s if given else None)
        if not given:  # as with torch's own operations in a stream's context
            g.record_stream(s)
            scale.record_stream(s)
        state, table = opt.state.numel(), opt._table.numel()
        del g, scale, opt
        for k in range(4):
            for size in (4 * n, state, table, 4):
                torch.full((size,), 77, dtype=torch.uint8, device=DEV)
        s.synchronize()
        assert torch.equal(p, ref)


def test_a_stream_given_by_its_pointer():
    say("operators on a raw stream")
    s = torch.cuda.Stream()
    p, g = torch.ones(300, device=DEV), torch.ones(300, device=DEV)
    x = torch.randn(2, 300, 8, device=DEV)
    torch.cuda.synchronize()
    for raw in (s.cuda_stream, torch.cuda.ExternalStream(s.cuda_stream)):
        opt = B.sla_adamw_create([p], stream=raw)
        B.sla_adamw_step(opt, [g], step=1, lr=1e-2, stream=raw)
        h, _, _ = B.sla_linrec_forward(x, x, stream=raw)
        s.synchronize()
        assert bool((p < 1).all()) and torch.equal(h, B.sla_linrec_forward(x, x)[0])


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_past_the_caches(bits):
    """A step that moves more than 256 MB reads and writes past the caches: its
    small tensors (partial blocks, any alignment, every type, bf16 copies) have
    the bits of a step of their own, which goes through them, and so have the
    ends of the large one."""
    say("adamw past the caches", bits)
    gen = torch.Generator(device=DEV).manual_seed(3)
    kinds = [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
             (torch.bfloat16, torch.bfloat16), (torch.float64, torch.float64)]
    parts, grads, low = [], [], []
    for k, n in enumerate([1, 3, 255, 256, 257, 1021, 4095, 4096, 10_000] * 4):
        pd, gd = kinds[k % 4]
        shift = k % 5
        parts.append(torch.randn(n + 8, device=DEV, generator=gen).to(pd)[shift:shift + n])
        grads.append(torch.randn(n + 8, device=DEV, generator=gen).to(gd)[k % 3:k % 3 + n])
        low.append(torch.zeros(n + 1, device=DEV, dtype=torch.bfloat16)[k % 2:k % 2 + n]
                   if pd == torch.float32 else None)
    n = 20_000_003
    big, gbig = torch.randn(n, device=DEV, generator=gen), torch.randn(n, device=DEV, generator=gen)

    def run(tail, gtail):
        ps = [torch.empty_like(torch.zeros(p.numel() + 8, device=DEV, dtype=p.dtype))
              [k % 5:k % 5 + p.numel()].copy_(p) for k, p in enumerate(parts)] + [tail.clone()]
        cs = [None if c is None else torch.zeros_like(c) for c in low] + [None]
        opt = B.sla_adamw_create(ps, state_bits=bits, grad_dtype=[g.dtype for g in grads] +
                                 [torch.float32], copies=cs)
        for t in (1, 2, 3):
            B.sla_adamw_step(opt, grads + [gtail], step=t, lr=1e-2, seed=9)
        return opt, ps, cs, B.sla_adamw_get_state(opt)

    head = 256 * 40
    big_opt, big_ps, big_cs, big_state = run(big, gbig)
    opt, ps, cs, state = run(big[:head], gbig[:head])
    for a, b in zip(big_ps[:-1] + [big_ps[-1][:head]] + big_cs, ps + cs):
        assert (a is None and b is None) or torch.equal(a, b)
    for a, b in zip(big_state, state):
        assert torch.equal(a[:opt.padded], b)
    # 32-bit states know no place, so the end can be compared as well
    if bits == 32:
        end = n // 256 * 256 - head
        _, ps, _, state = run(big[end:], gbig[end:])
        assert torch.equal(big_ps[-1][end:], ps[-1])
        for a, b in zip(big_state, state):
            size = n - end
            at, small = big_opt.starts[-1] + end, opt.starts[-1]
            assert torch.equal(a[at:at + size], b[small:small + size])


@pytest.mark.parametrize("bits", [32, 8])
def test_states_read_through_the_c_entry(bits):
    """sla_adamw_get_state copies 32-bit states out as well."""
    say("adamw states in C", bits)
    p, g = torch.randn(3000, device=DEV), torch.randn(3000, device=DEV)
    opt = B.sla_adamw_create([p], state_bits=bits)
    B.sla_adamw_step(opt, [g], step=1, lr=1e-2)
    want = B.sla_adamw_get_state(opt)
    out = [torch.full_like(t, 7.0) for t in want]
    raw = torch.cuda.current_stream().cuda_stream
    assert B.lib().sla_adamw_get_state(opt.handle, out[0].data_ptr(), out[1].data_ptr(), raw) == 0
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert B.lib().sla_adamw_get_state(opt.handle, out[0].data_ptr(), out[0].data_ptr(), raw) == -1
    state, table, padded = B.sla_adamw_sizes([p], bits)
    assert (state, padded) == (opt.state.numel(), opt.padded) and table == opt._table.numel()

"""The AdamW step over many tensors against plain computations: 8-bit codes
bit for bit, states and parameters in 32 bits within a few roundings."""
import numpy as np
import pytest
import torch

from preconditioned_cg_solver_amd import binding as B
from gpu_util import DEV, say
import seq_util as S

pytestmark = pytest.mark.gpu

HY = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
DT = {"f64": torch.float64, "f32": torch.float32, "bf16": torch.bfloat16}
SIZES = [1, 3, 255, 256, 257, 0, 4095, 4096, 4097, 10_000]


def host(t):
    return t.detach().double().cpu().numpy()


def make(pd, gd, sizes, seed):
    r = np.random.default_rng([11, seed, len(sizes)])
    ps = [torch.from_numpy(0.1 * r.standard_normal(n)).to(DT[pd]).to(DEV) for n in sizes]
    gs = [torch.from_numpy(1e-3 * np.exp(2 * r.standard_normal(n)) * r.standard_normal(n))
          .to(DT[gd]).to(DEV) for n in sizes]
    return ps, gs


def padded(gs):
    """float32 gradients in the padded order."""
    return S.pad_to_blocks([g.detach().float().cpu().numpy() for g in gs])


def starting_states(n, seed):
    r = np.random.default_rng([12, seed])
    m = (1e-3 * r.standard_normal(n)).astype(np.float32)
    v = (1e-6 * np.exp(2 * r.standard_normal(n))).astype(np.float32)
    return m, v


def real_places(sizes):
    return S.pad_to_blocks([np.ones(n) for n in sizes]) > 0


def check_params(ps, before, m0, v0, gs, sizes, step, pd, copies=None):
    """p within the roundings of its update: 12 of fp32 on the update's terms
    (m', v', root, quotient; the state's own products and sums), 4 on p, and
    the storage type's."""
    at = 0
    for k, (p, b, g, n) in enumerate(zip(ps, before, gs, sizes)):
        sl = slice(at, at + n)
        at += -(-n // 256) * 256
        gg = g.detach().float().double().cpu().numpy()
        want, m1, v1, up = S.adamw64(b, m0[sl].astype(np.float64), v0[sl].astype(np.float64), gg,
                                     step, HY["lr"], HY["beta1"], HY["beta2"], HY["eps"],
                                     HY["weight_decay"])
        terms = HY["lr"] / (1 - HY["beta1"] ** step) * \
            (np.abs(HY["beta1"] * m0[sl]) + np.abs((1 - HY["beta1"]) * gg)) / \
            (np.sqrt(v1 / (1 - HY["beta2"] ** step)) + HY["eps"])
        bound = 12 * S.U32 * terms
        own = {"f64": 4 * S.U64, "f32": 4 * S.U32, "bf16": 2.0 ** -7}[pd]  # bf16: up or down a step
        bound = bound + own * (np.abs(b) + np.abs(up))
        off = np.abs(host(p) - want)
        assert np.all(off <= bound), (k, n, float(np.max(off / np.maximum(bound, 1e-300))))
        if copies is not None:
            assert torch.equal(copies[k], p.to(torch.bfloat16))


@pytest.mark.parametrize("pd,gd", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"),
                                   ("f64", "f64")])
@pytest.mark.parametrize("bits", [32, 8])
def test_steps(pd, gd, bits):
    say("adamw", pd, gd, bits)
    ps, gs = make(pd, gd, SIZES, 1)
    opt = B.sla_adamw_create(ps, state_bits=bits, grad_dtype=DT[gd])
    m, v = starting_states(opt.padded, 1)
    real = real_places(SIZES)
    m, v = np.where(real, m, 0).astype(np.float32), np.where(real, v, 0).astype(np.float32)
    B.sla_adamw_set_state(opt, torch.from_numpy(m).to(DEV), torch.from_numpy(v).to(DEV))
    m, v = (host(t).astype(np.float32) for t in B.sla_adamw_get_state(opt))
    for step in (5, 6, 7):
        before = [host(p) for p in ps]
        B.sla_adamw_step(opt, gs, step=step, seed=99, **HY)
        gm, gv = (host(t) for t in B.sla_adamw_get_state(opt))
        check_params(ps, before, m, v, gs, SIZES, step, pd)
        m, v = S.moments32(m, v, padded(gs), HY["beta1"], HY["beta2"])
        if bits == 8:
            r = S.noise(99, step, opt.padded)
            m = S.levels(m, ((r & np.uint64(0xFFFF)) << np.uint64(4)) + np.uint64(8), 126, 0)
            v = S.levels(v, ((r >> np.uint64(16)) << np.uint64(4)) + np.uint64(8), 254, 1)
        assert np.array_equal(gm, m.astype(np.float64)) and np.array_equal(gv, v)
        gs = [(-0.7 * g.double()).to(g.dtype) for g in gs]


def test_bf16_rounding_is_the_documented_one():
    say("adamw bf16 rounding")
    ps, gs = make("bf16", "bf16", [5000], 2)
    before = ps[0].float().cpu().numpy()
    opt = B.sla_adamw_create(ps, state_bits=32)
    B.sla_adamw_step(opt, gs, step=1, seed=3 + (1 << 40), **HY)
    want, _, _, _ = S.adamw64(before.astype(np.float64), 0.0, 0.0, host(gs[0]), 1, HY["lr"],
                              HY["beta1"], HY["beta2"], HY["eps"], HY["weight_decay"])
    r = S.mix(S.noise(3 + (1 << 40), 1, 5000) + np.uint64(0x6A09E667)) & np.uint64(0xFFFF)
    bits = want.astype(np.float32).view(np.uint32).astype(np.uint64)
    low = bits & np.uint64(0xFFFF)
    up = (((bits + r) >> np.uint64(16)) << np.uint64(16)).astype(np.uint32).view(np.float32)
    # fp32 rounding of the update moves the remainder by a few units of 2^-16
    sure = np.abs((low + r).astype(np.int64) - 65536) > 64
    assert sure.mean() > 0.99
    assert np.array_equal(ps[0].float().cpu().numpy()[sure], up[sure])


def test_rounding_is_unbiased():
    """One step moves v by 0.1 % of levels 12 % apart: the mean over elements
    follows the exact value.  With probabilities q of rounding up a level the
    mean of n values is off by at most 5 sqrt(q (1 - q) / n) levels with
    probability 1 - 6e-7."""
    say("adamw unbiased rounding")
    n = 1 << 20
    p, g = torch.zeros(n, device=DEV), torch.full((n,), 1.5e-3, device=DEV)
    opt = B.sla_adamw_create([p], state_bits=8)
    m, v = torch.full((n,), 1e-3, device=DEV), torch.full((n,), 1.1e-6, device=DEV)
    # each block's largest element fixes the levels
    m[::256], v[::256] = 4e-3, 9e-6
    B.sla_adamw_set_state(opt, m, v)
    m, v = (t.clone() for t in B.sla_adamw_get_state(opt))
    B.sla_adamw_step(opt, [g], step=10, seed=5, **HY)
    m2, v2 = B.sla_adamw_get_state(opt)
    for old, new, b, add in ((m, m2, 0.9, 1.5e-3), (v, v2, 0.999, 1.5e-3 ** 2)):
        want = b * float(old[1]) + (1 - b) * add
        inner = host(new).reshape(-1, 256)[:, 1:]
        lo = 2.0 ** np.floor(np.log2(want))
        level = lo / 8
        q = (want - lo) / level % 1.0
        bound = 5 * np.sqrt(q * (1 - q) / inner.size) * level + 2.0 ** -16 * level
        assert abs(inner.mean() - want) <= bound, (inner.mean(), want, q)
        assert np.all(np.abs(inner - want) < level)


def test_states_survive_a_round_trip():
    say("adamw state round trip")
    sizes = [700, 3, 256 * 9]
    ps, gs = make("f32", "f32", sizes, 3)
    a = B.sla_adamw_create(ps, state_bits=8)
    for step in (1, 2, 3):
        B.sla_adamw_step(a, gs, step=step, **HY)
    m, v = B.sla_adamw_get_state(a)
    b = B.sla_adamw_create([p.clone() for p in ps], state_bits=8)
    B.sla_adamw_set_state(b, m.float(), v.float())
    m2, v2 = B.sla_adamw_get_state(b)
    assert torch.equal(m, m2) and torch.equal(v, v2)
    parts = a.views(m)
    assert [t.shape for t in parts] == [p.shape for p in ps]
    # bytes: save and resume
    keep, held = a.state.clone(), [p.clone() for p in ps]
    B.sla_adamw_step(a, gs, step=4, **HY)
    after = [p.clone() for p in ps], a.state.clone()
    assert not torch.equal(keep, a.state)
    a.state.copy_(keep)
    for p, q in zip(ps, held):
        p.copy_(q)
    B.sla_adamw_step(a, gs, step=4, **HY)
    assert torch.equal(a.state, after[1]) and all(map(torch.equal, ps, after[0]))
    # nearest level: within half a level (1/16); below a block's range (2^-15
    # of its largest for m, 2^-31 for v) zero or the lowest level
    r = np.random.default_rng(4)
    x = np.exp(3 * r.standard_normal(a.padded)).astype(np.float32)
    x[~real_places(sizes)] = 0
    B.sla_adamw_set_state(b, torch.from_numpy(x).to(DEV), torch.from_numpy(x).to(DEV))
    largest = np.repeat(x.reshape(-1, 256).max(1), 256)
    for t, reach in zip(B.sla_adamw_get_state(b), (2.0 ** -15, 2.0 ** -31)):
        assert np.all(np.abs(host(t) - x) <= np.maximum(x / 16, largest * reach))


def test_small_and_large_values_in_one_block():
    """v below the block's range is held at the lowest level, not at zero (a
    zero would make the next update huge); m below it becomes zero."""
    say("adamw range of a block")
    p = torch.zeros(256, device=DEV)
    opt = B.sla_adamw_create([p], state_bits=8)
    g = torch.full((256,), 1e-12, device=DEV)
    g[0] = 1.0
    B.sla_adamw_step(opt, [g], step=1, lr=1.0, eps=0.0, weight_decay=0.0)
    m, v = (host(t) for t in B.sla_adamw_get_state(opt))
    assert np.all(v[1:] > 0) and np.all(v[1:] < v[0] * 2.0 ** -30)
    assert np.all(m[1:] == 0) and abs(m[0] - 0.1) <= 0.1 / 8
    # this step's update used the unrounded values: sign(g) lr
    assert np.all(np.abs(host(p) + 1.0) <= 1e-5)


def test_non_finite_gradients_stay_in_their_element():
    for bits in (32, 8):
        say("adamw non-finite", bits)
        ps, gs = make("f32", "f32", [1000], 6)
        clean = [p.clone() for p in ps]
        gs[0][10], gs[0][300] = float("nan"), float("inf")
        same = [g.clone() for g in gs]
        same[0][10] = same[0][300] = 0.0
        opt, ref = (B.sla_adamw_create(q, state_bits=bits) for q in (ps, clean))
        for step in (1, 2):
            B.sla_adamw_step(opt, gs, step=step, **HY)
            B.sla_adamw_step(ref, same, step=step, **HY)
        m, v = (host(t)[:1000] for t in B.sla_adamw_get_state(opt))
        rm, rv = (host(t)[:1000] for t in B.sla_adamw_get_state(ref))
        ok = np.ones(1000, bool)
        ok[[10, 300]] = False
        assert not np.isfinite(m[10]) and not np.isfinite(m[300])
        assert not np.isfinite(v[10]) and not np.isfinite(v[300])
        assert np.array_equal(m[ok], rm[ok]) and np.array_equal(v[ok], rv[ok])
        assert np.array_equal(host(ps[0])[ok], host(clean[0])[ok])


def test_gradient_scale():
    say("adamw gradient scale")
    ps, gs = make("f32", "bf16", [777, 40], 7)
    qs = [p.clone() for p in ps]
    a = B.sla_adamw_create(ps, state_bits=8, grad_dtype=torch.bfloat16)
    b = B.sla_adamw_create(qs, state_bits=8)
    B.sla_adamw_step(a, gs, step=1, seed=1, grad_scale=torch.tensor([0.37], device=DEV), **HY)
    B.sla_adamw_step(b, [g.float() * 0.37 for g in gs], step=1, seed=1, **HY)
    assert all(torch.equal(p, q) for p, q in zip(ps, qs)) and torch.equal(a.state, b.state)
    held, old = a.state.clone(), [p.clone() for p in ps]
    for bad in (float("nan"), float("inf")):
        B.sla_adamw_step(a, gs, step=2, grad_scale=torch.tensor(bad, device=DEV), **HY)
    assert torch.equal(held, a.state) and all(torch.equal(p, q) for p, q in zip(ps, old))


def test_missing_gradients_and_copies():
    say("adamw None gradients, bf16 copies")
    ps, gs = make("f32", "f32", [300, 513, 5], 8)
    copies = [torch.zeros_like(p, dtype=torch.bfloat16) for p in ps]
    opt = B.sla_adamw_create(ps, copies=copies)
    old = [p.clone() for p in ps]
    B.sla_adamw_step(opt, [gs[0], None, gs[2]], step=1, **HY)
    m, _ = B.sla_adamw_get_state(opt)
    parts = opt.views(m)
    assert torch.equal(ps[1], old[1]) and float(parts[1].abs().sum()) == 0.0
    assert float(copies[1].abs().sum()) == 0.0
    for k in (0, 2):
        assert not torch.equal(ps[k], old[k]) and torch.equal(copies[k], ps[k].bfloat16())


def test_mixed_types_and_many_tensors():
    """Every type pair in one handle, and more tensors than one launch takes."""
    say("adamw mixed, 1000 tensors")
    kinds = [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f64", "f64")]
    sizes = [(37 * k) % 900 for k in range(1000)]
    r = np.random.default_rng(9)
    ps, gs, each = [], [], []
    for k, n in enumerate(sizes):
        pd, gd = kinds[(k // 3) % 4] if k < 500 else kinds[0]
        ps.append(torch.from_numpy(r.standard_normal(n)).to(DT[pd]).to(DEV))
        gs.append(torch.from_numpy(r.standard_normal(n)).to(DT[gd]).to(DEV))
        each.append(pd)
    before = [host(p) for p in ps]
    opt = B.sla_adamw_create(ps, grad_dtype=[g.dtype for g in gs])
    B.sla_adamw_step(opt, gs, step=1, **HY)
    zero = np.zeros(opt.padded, np.float32)
    at = 0
    for p, b, g, n, pd in zip(ps, before, gs, sizes, each):
        pad = -(-n // 256) * 256
        check_params([p], [b], zero[:pad], zero[:pad], [g], [n], 1, pd)
        at += pad
    gm, gv = (host(t) for t in B.sla_adamw_get_state(opt))
    m, v = S.moments32(zero, zero, padded(gs), 0.9, 0.999)
    assert np.array_equal(gm, m) and np.array_equal(gv, v)


@pytest.mark.parametrize("pd", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_parameters_at_any_element(pd, bits):
    """Slices that begin at every residue of a 16-byte line equal whole tensors."""
    say("adamw misaligned", pd, bits)
    n = 3000
    flat = torch.zeros(n + 16, dtype=DT[pd], device=DEV)
    gflat = torch.zeros(n + 16, dtype=DT[pd], device=DEV)
    (p0,), (g0,) = make(pd, pd, [n], 10)
    ref = p0.clone()
    o = B.sla_adamw_create([ref], state_bits=bits)
    B.sla_adamw_step(o, [g0], step=1, seed=4, **HY)
    for shift in (0, 1, 2, 3, 4, 7):
        for gshift in (0, 1):
            flat.fill_(7)
            p, g = flat[shift:shift + n], gflat[gshift:gshift + n]
            p.copy_(p0)
            g.copy_(g0)
            a = B.sla_adamw_create([p], state_bits=bits)
            B.sla_adamw_step(a, [g], step=1, seed=4, **HY)
            assert torch.equal(p, ref) and torch.equal(a.state, o.state), (shift, gshift)
            assert torch.all(flat[:shift] == 7) and torch.all(flat[shift + n:] == 7)


def test_no_tensors():
    say("adamw without tensors")
    opt = B.sla_adamw_create([])
    B.sla_adamw_step(opt, [], step=1, lr=1e-3)
    e = B.sla_adamw_create([torch.zeros(0, device=DEV)], state_bits=8)
    B.sla_adamw_step(e, [torch.zeros(0, device=DEV)], step=1, lr=1e-3)
    m, v = B.sla_adamw_get_state(e)
    assert m.numel() == v.numel() == 0


def test_captured_in_a_graph():
    """Each replay makes one more step with the captured step number."""
    say("adamw in a graph")
    ps, gs = make("f32", "f32", [5000, 17], 13)
    qs = [p.clone() for p in ps]
    a, b = B.sla_adamw_create(ps, state_bits=8), B.sla_adamw_create(qs, state_bits=8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sla_adamw_step(a, gs, step=3, seed=2, **HY)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        B.sla_adamw_step(b, gs, step=3, seed=2, **HY)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ps, qs)) and torch.equal(a.state, b.state)
        for g in gs:
            g.mul_(-0.9)


def test_on_another_stream():
    say("adamw on a side stream")
    ps, gs = make("f32", "f32", [5000], 14)
    before = [host(p) for p in ps]
    s = torch.cuda.Stream()
    opt = B.sla_adamw_create(ps, stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.ones(1 << 26, device=DEV)
        for _ in range(20):
            big.mul_(1.0)
        gs2 = [g * big[0] for g in gs]
    B.sla_adamw_step(opt, gs2, step=1, stream=s, **HY)
    s.synchronize()
    zero = np.zeros(opt.padded, np.float32)
    check_params(ps, before, zero, zero, gs, [5000], 1, "f32")


def test_quadratic_is_minimised_as_well_in_8_bits():
    """A quadratic with curvatures over three decades, noisy gradients: the
    8-bit run ends within a factor of two of the 32-bit run's loss."""
    say("adamw quadratic")
    n = 4096
    c = torch.logspace(-1, 2, n, device=DEV)
    loss = {}
    for bits in (32, 8):
        gen = torch.Generator(device=DEV).manual_seed(1)
        p = torch.randn(n, device=DEV, generator=gen)
        opt = B.sla_adamw_create([p], state_bits=bits)
        for t in range(1, 401):
            g = c * p + 0.1 * torch.randn(n, device=DEV, generator=gen)
            B.sla_adamw_step(opt, [g], step=t, lr=2e-2 * (1 - t / 401), weight_decay=0.0, seed=7)
        loss[bits] = float((c * p * p).mean())
    assert loss[8] <= 2 * loss[32], loss

"""The operators of a sequence block together and through autograd, on streams and in
graphs, and the study that learns one."""
import numpy as np
import pytest
import torch

from preconditioned_cg_solver_amd import autograd as AG
from preconditioned_cg_solver_amd import binding as B
from preconditioned_cg_solver_amd import studies
from block_gpu import DT, make, own_of
from gpu_util import say

pytestmark = pytest.mark.gpu


def parameters(r, width, states, dtype):
    p = {"norm": r.own(width), "split": r(width, 2 * width), "conv": r.own(width, 4),
         "conv_bias": r.own(width), "drive": r(width, width + 2 * states) * 0.2,
         "rate": r.own(width, states).abs(), "skip": r.own(width), "dt_bias": r.own(width) - 2,
         "gated": r.own(width), "scale": r.own(width)}
    p["split"] = p["split"] / width ** 0.5
    return {k: v.requires_grad_() for k, v in p.items()}


def block(p, stream, offsets=None, conv_state=None, h0=None):
    """norm -> projection -> convolution -> scan -> gated norm onto the stream."""
    width, states = p["rate"].shape
    y, stream = AG.norm_in(stream, p["norm"])
    x, gate = (y @ p["split"]).split(width, -1)
    x, tail = AG.causal_conv(x, p["conv"], p["conv_bias"], state=conv_state, offsets=offsets)
    dt, b, c = (x @ p["drive"]).split([width, states, states], -1)
    y, last = AG.selective_scan(x, dt, -p["rate"], b.unsqueeze(-2), c.unsqueeze(-2), D=p["skip"],
                                dt_bias=p["dt_bias"], h0=h0, offsets=offsets)
    return AG.norm_out(y, p["gated"], gate=gate, residual=stream, scale=p["scale"]), tail, last


def plain(p, stream, offsets=None, conv_state=None, h0=None, eps=1e-5):
    """The same of elementary operations, for torch to differentiate."""
    width, states = p["rate"].shape

    def normed(v):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps)

    y = normed(stream) * p["norm"]
    xs, gate = (y @ p["split"]).split(width, -1)
    bounds = [(s, None, None) for s in range(stream.shape[0])] if offsets is None else \
        [(None, a, b) for a, b in zip(offsets.tolist(), offsets.tolist()[1:])]
    outs, tails, lasts = [], [], []
    for i, (s, a, b) in enumerate(bounds):
        x = xs[s] if offsets is None else xs[a:b]
        head = x.new_zeros(3, width) if conv_state is None else conv_state[i]
        row = torch.cat([head, x])
        pre = p["conv_bias"] + sum(row[j:j + len(x)] * p["conv"][:, j] for j in range(4))
        tails.append(row[len(x):])
        x = pre * torch.sigmoid(pre)
        dt, bs, cs = (x @ p["drive"]).split([width, states, states], -1)
        delta = torch.nn.functional.softplus(dt + p["dt_bias"])
        h = x.new_zeros(width, states) if h0 is None else h0[i]
        ys = []
        for t in range(len(x)):
            h = torch.exp(delta[t, :, None] * -p["rate"]) * h + \
                (delta[t] * x[t])[:, None] * bs[t]
            ys.append((h * cs[t]).sum(1) + p["skip"] * x[t])
        lasts.append(h)
        outs.append(torch.stack(ys) if ys else x)
    y = torch.stack(outs) if offsets is None else torch.cat(outs)
    n = normed(y * (gate * torch.sigmoid(gate))) * p["gated"]
    return stream + p["scale"] * n, torch.stack(tails), torch.stack(lasts)


def loss_of(outs, weights):
    return sum((o.double() * w).sum() for o, w in zip(outs, weights))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", ["f64", "f32"])
def test_block_against_elementary_operations(dtype, packed):
    """Outputs and all gradients: in fp64 to 1e-9; in fp32 to 2e-4 of the gradient's size, some
    300 roundings of 2^-24 through five operators whose factors here are of order 10."""
    say("block", dtype, packed)
    r = make(0, dtype)
    width, states = 24, 16
    off = torch.tensor([0, 7, 7, 40, 41, 66], device="cuda") if packed else None
    lead, n = ((66,), 5) if packed else ((2, 33), 2)
    p = parameters(r, width, states, dtype)
    extra = {"stream": r(*lead, width).requires_grad_(),
             "conv_state": r(n, 3, width).requires_grad_(),
             "h0": r.own(n, width, states).requires_grad_()}
    outs = block(p, offsets=off, **extra)
    q = {k: v.detach().double().requires_grad_() for k, v in {**p, **extra}.items()}
    ref = plain({k: q[k] for k in p}, offsets=off, **{k: q[k] for k in extra})
    weights = [torch.randn_like(o) for o in ref]
    tol = 1e-9 if dtype == "f64" else 2e-4
    for a, b in zip(outs, ref):
        assert (a - b).norm() <= tol * b.norm()
    got = torch.autograd.grad(loss_of(outs, weights), [*p.values(), *extra.values()])
    want = torch.autograd.grad(loss_of(ref, weights), list(q.values()))
    for name, a, b in zip(q, got, want):
        assert (a - b).norm() <= tol * b.norm(), name


def test_block_in_bf16_runs_and_is_near():
    """bf16 between the operators: within 5% of the fp64 block of the same parameters, by norm (some
    ten roundings of 2^-8 in a row, factors of order one)."""
    r = make(1, "bf16")
    p = parameters(r, 64, 16, "bf16")
    p["drive"] = p["drive"].detach().requires_grad_()
    stream = r(2, 100, 64).requires_grad_()
    outs = block(p, stream)
    assert outs[0].dtype == torch.bfloat16 and outs[2].dtype == torch.float32
    q = {k: v.detach().double() for k, v in p.items()}
    ref = plain(q, stream.detach().double())
    assert (outs[0].double() - ref[0]).norm() <= 0.05 * ref[0].norm()
    grads = torch.autograd.grad(outs[0].float().square().mean(), [stream, *p.values()])
    assert all(torch.isfinite(g).all() for g in grads)
    assert [g.dtype for g in grads] == [t.dtype for t in (stream, *p.values())]


def test_prefill_then_tokens_is_the_whole():
    """A prompt, then single tokens with the states it left, in place."""
    r = make(2, "f32")
    p = parameters(r, 32, 16, "f32")
    stream = r(3, 50, 32)
    with torch.no_grad():
        whole, tail, last = block(p, stream)
        out, cs, hs = block(p, stream[:, :37].contiguous())
        outs = [out]
        for t in range(37, 50):
            y, s = AG.norm_in(stream[:, t:t + 1], p["norm"])
            x, gate = (y @ p["split"]).split(32, -1)
            x, _ = B.sla_conv_forward(x, p["conv"], bias=p["conv_bias"], state=cs, last=cs)
            dt, b, c = (x @ p["drive"]).split([32, 16, 16], -1)
            y, _, _ = B.sla_selscan_forward(x, dt, -p["rate"], b.unsqueeze(2), c.unsqueeze(2),
                                            D=p["skip"], dt_bias=p["dt_bias"], h0=hs, h_last=hs)
            outs.append(AG.norm_out(y, p["gated"], gate=gate, residual=s, scale=p["scale"]))
    assert torch.allclose(torch.cat(outs, 1), whole, rtol=1e-3, atol=1e-3)
    assert torch.allclose(hs, last, rtol=1e-3, atol=1e-4)
    assert torch.allclose(cs, tail, rtol=1e-3, atol=1e-4)


def test_gradients_that_are_missing_or_expanded():
    r = make(3, "f32")
    x, w = r(2, 9, 8).requires_grad_(), r.own(8, 4).requires_grad_()
    y, last = AG.causal_conv(x, w)
    a = torch.autograd.grad(y.sum(), [x, w], retain_graph=True)  # an expanded gradient
    b = torch.autograd.grad((y * torch.ones_like(y)).sum(), [x, w])
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    y, last = AG.causal_conv(x, w)
    g, = torch.autograd.grad(last.sum(), x)
    assert g[:, -3:].eq(1).all() and not g[:, :-3].any()
    A, bc = -r.own(8, 4).abs(), r(2, 9, 1, 4)
    y, last = AG.selective_scan(x, x, A, bc, bc)
    g1, = torch.autograd.grad(last.sum(), x, retain_graph=True)
    g2, = torch.autograd.grad(last.sum() + 0 * y.sum(), x)
    assert torch.equal(g1, g2)
    v = r.own(8).requires_grad_()
    y, s = AG.norm_in(x, v, residual=r(2, 9, 8))
    g, = torch.autograd.grad(s.sum(), x)
    assert g.eq(1).all()
    y, s = AG.norm_in(x, v)
    assert s is x
    torch.autograd.grad(y.sum(), [x, v])
    # a parameter used twice has both gradients
    y1, _ = AG.norm_in(x, v)
    y2, _ = AG.norm_in(y1, v)
    g, = torch.autograd.grad(y2.sum(), v)
    assert torch.isfinite(g).all()


def test_gradients_are_differentiable_once_and_see_changes():
    r = make(4, "f32")
    x, w = r(1, 5, 8).requires_grad_(), r.own(8, 4).requires_grad_()
    y, _ = AG.causal_conv(x, w)
    g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), x)
    h0 = r.own(1, 8, 4).requires_grad_()
    A, bc = -r.own(8, 4).abs(), r(1, 5, 1, 4)
    held = h0.detach().clone()
    y, _ = AG.selective_scan(x, x, A, bc, bc, h0=held)
    B.sla_selscan_forward(x.detach(), x.detach(), A, bc, bc, h0=held, h_last=held)
    with pytest.raises(RuntimeError):  # the saved state has been overwritten
        y.sum().backward()


def everything(t):
    """One pass of each operator, forward and backward."""
    y, last = B.sla_conv_forward(t["x"], t["w"], bias=t["v"], state=t["cs"])
    out = [y, last, *B.sla_conv_backward(t["x"], t["w"], t["dy"], bias=t["v"], state=t["cs"])]
    first = (t["x"], t["dt"], t["A"], t["B"], t["C"])
    rest = dict(D=t["v"], z=t["z"], dt_bias=t["v"], h0=t["h0"])
    y, last, saved = B.sla_selscan_forward(*first, **rest, save=True)
    out += [y, last, saved, *B.sla_selscan_backward(*first, saved, t["dy"], **rest)]
    y, r, rstd = B.sla_norm_in_forward(t["x"], t["v"], residual=t["z"], scale=t["v"])
    out += [y, r, *B.sla_norm_in_backward(t["dy"], t["x"], t["v"], rstd, residual=t["z"],
                                          scale=t["v"], grad_r=t["z"])]
    y, rstd = B.sla_norm_out_forward(t["x"], t["v"], gate=t["z"], residual=t["dt"])
    out += [y, *B.sla_norm_out_backward(t["dy"], t["x"], t["v"], rstd, gate=t["z"])]
    return [o for o in out if o is not None]


def tensors(seed, dtype="bf16", n=2, steps=300, d=40):
    r = make(seed, dtype)
    return {"x": r(n, steps, d), "dt": r(n, steps, d), "z": r(n, steps, d), "dy": r(n, steps, d),
            "B": r(n, steps, 1, 16), "C": r(n, steps, 1, 16), "w": r.own(d, 4), "v": r.own(d),
            "cs": r(n, 3, d), "A": -r.own(d, 16).abs(), "h0": r.own(n, d, 16)}


def test_on_another_stream():
    t = tensors(5)
    want = everything(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = everything(t)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # given by argument
    side.wait_stream(torch.cuda.current_stream())
    y, last = B.sla_conv_forward(t["x"], t["w"], bias=t["v"], state=t["cs"], stream=side)
    s, hl, _ = B.sla_selscan_forward(t["x"], t["dt"], t["A"], t["B"], t["C"], stream=side)
    n, _, _ = B.sla_norm_in_forward(t["x"], t["v"], stream=side)
    o, _ = B.sla_norm_out_forward(t["x"], t["v"], gate=t["z"], stream=side)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(last, want[1])
    assert torch.equal(s, B.sla_selscan_forward(t["x"], t["dt"], t["A"], t["B"], t["C"])[0])
    assert torch.equal(n, B.sla_norm_in_forward(t["x"], t["v"])[0])
    assert torch.equal(o, B.sla_norm_out_forward(t["x"], t["v"], gate=t["z"])[0])


def test_two_calls_at_once():
    """On two streams, with workspaces of their own: the results of one after the other."""
    ts = [tensors(6), tensors(7)]
    want = [everything(t) for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(3):
        got = []
        for t, s in zip(ts, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(everything(t))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_captured_and_replayed():
    """Two graphs of the operators, replayed in turn with other inputs and eager work between."""
    graphs = []
    for seed in (8, 9):
        t = tensors(seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            everything(t)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = everything(t)
        graphs.append((g, t, out))
    for turn in range(4):
        for g, t, out in graphs:
            fresh = tensors(20 + turn)
            for k in t:
                t[k].copy_(fresh[k])
            g.replay()
            torch.cuda.synchronize()
            want = everything(fresh)
            assert all(torch.equal(a, b) for a, b in zip(out, want)), turn


def test_rows_past_the_caches():
    """Calls of more than 256 MB, which go past the last-level cache: the same bits as calls of
    a part, and the weights' gradients as the sum of the parts' to fp32 rounding."""
    r = make(10, "bf16")
    n, steps, d = 8, 4096, 4096
    x, z = r(n, steps, d), r(n, steps, d)
    w, v = r.own(d, 4), r.own(d)
    y, _ = B.sla_conv_forward(x, w)
    assert torch.equal(y[:1], B.sla_conv_forward(x[:1], w)[0])
    dx, dw, _, _ = B.sla_conv_backward(x, w, z)
    parts = [B.sla_conv_backward(x[k:k + 1], w, z[k:k + 1]) for k in range(n)]
    assert torch.equal(dx[3:4], parts[3][0])
    total = sum(p[1].double() for p in parts)
    assert (dw - total).norm() <= 1e-5 * total.norm()
    y, s, rstd = B.sla_norm_in_forward(x, v, residual=z, scale=v)
    y1, s1, r1 = B.sla_norm_in_forward(x[:1], v, residual=z[:1], scale=v)
    assert torch.equal(y[:1], y1) and torch.equal(s[:1], s1) and torch.equal(rstd[:1], r1)
    g = B.sla_norm_in_backward(x, x, v, rstd, residual=z, scale=v)
    g1 = B.sla_norm_in_backward(x[:1], x[:1], v, r1, residual=z[:1], scale=v)
    assert torch.equal(g[0][:1], g1[0]) and torch.equal(g[1][:1], g1[1])
    o, rstd = B.sla_norm_out_forward(x, v, gate=z)
    o1, r1 = B.sla_norm_out_forward(x[:1], v, gate=z[:1])
    assert torch.equal(o[:1], o1)
    g = B.sla_norm_out_backward(x, x, v, rstd, gate=z)
    g1 = B.sla_norm_out_backward(x[:1], x[:1], v, r1, gate=z[:1])
    assert torch.equal(g[0][:1], g1[0]) and torch.equal(g[1][:1], g1[1])


def test_the_study_with_a_block_runs():
    out = studies.learn(iters=5, sources="block")
    assert np.isfinite(out["loss_last"]) and out["parameters"] > 4096
    with pytest.raises(ValueError):
        studies.learn(iters=1, sources="other")


def test_the_blocks_gradients_through_a_readout():
    """block_sources' gradients against central differences along a random direction."""
    p = studies.block_parameters(50, width=16, states=4)
    drive = torch.cumsum(torch.randn(30, dtype=torch.float64, device="cuda"), 0) / 4
    weight = torch.randn(30, 50, dtype=torch.float64, device="cuda")

    def loss(q):
        return (studies.block_sources(q, drive) * weight).sum()

    grads = torch.autograd.grad(loss(p), list(p.values()))
    for (name, t), g in zip(p.items(), grads):
        v, h = torch.randn_like(t), 1e-6
        with torch.no_grad():
            up, down = dict(p), dict(p)
            up[name], down[name] = t + h * v, t - h * v
            diff = float((loss(up) - loss(down)) / (2 * h))
        assert abs(diff - float((g * v).sum())) <= 1e-5 * (1 + abs(diff)), name


@pytest.mark.parametrize("dtype", [torch.float64, torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("marks", [[0, 70], [9, 9], [0, 31, 31, 61], [12, 40, 70], [70, 70], [7]])
def test_outputs_of_padded_rows_are_zeros(dtype, marks):
    """Memory that held NaN is handed out again: rows of no sequence are zeros all the same,
    so that what follows may sum over them."""
    wide = torch.float64 if dtype == torch.float64 else torch.float32
    gen = torch.Generator().manual_seed(4)

    def r(*s, t=dtype):
        return torch.randn(*s, generator=gen, dtype=torch.float64).to(t).cuda()

    x, dt, b = r(70, 23), r(70, 23), r(70, 1, 16)
    w, A = r(23, 4, t=wide), -r(23, 16, t=wide).abs()
    off = torch.tensor(marks, device="cuda")
    outside = torch.ones(70, dtype=torch.bool)
    outside[marks[0]:marks[-1]] = False
    for f in (lambda: B.sla_conv_forward(x, w, offsets=off),
              lambda: B.sla_selscan_forward(x, dt, A, b, b, offsets=off)):
        dirty = [torch.full((70, 23), float("nan"), dtype=dtype, device="cuda") for _ in range(8)]
        del dirty
        y = f()[0].cpu()
        assert torch.isfinite(y).all() and not y[outside].any()
    # in C: those rows and no others
    y = torch.full((70, 23), float("nan"), dtype=dtype, device="cuda")
    B.sla_rows_clear(y, off)
    y = y.cpu()
    assert not y[outside].any() and torch.isnan(y[~outside]).all()

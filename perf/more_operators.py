"""Measured cases of the causal convolution, the selective scan and the norms
of a sequence block.

  conv      y_t = act(b + sum_k w_k x_{t-K+1+k}), per channel, act the identity or silu
  scan      delta = softplus(dt + bias),  a = exp(delta A),  h_t = a h_{t-1} + delta x_t B_t,
            s_t = C_t . h_t + D x_t,  y_t = s_t silu(z_t), N states per channel
  norm_in   r = residual + scale x,  y = r / rms(r) weight
  norm_out  n = u / rms(u) weight with u = x silu(gate), or n = x / rms(x) weight silu(gate);
            out = residual + scale n

with rms(v) = sqrt(mean(v^2) + eps) along a row, and the gradients of each.
Sequences are dense (sequences, steps, channels) or packed (steps, channels)
with offsets; parameters and the scan's states are float32.

``own`` false: elementary torch operations in 32 bits, rounded once at the
end; ``own`` true: the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


# ----- cases -----

def listed():
    return [
        # serving: the next token of 32 sequences
        conv("conv_step_bf16", "step", "bf16", 32, 1, 4096, 4),
        # an ordinary training step; x is half of a fused projection
        conv("conv_train_bf16", "train", "bf16", 8, 2048, 2048, 4, fused=True),
        # packed sequences of very different lengths, an odd number of channels, full precision
        conv("conv_packed_f32_train", "train", "f32", 120, 50_003, 777, 3, packed=True, state=True),
        # serving: the next token of 16 sequences
        scan("scan_step_bf16", "step", "bf16", 16, 1, 4096, 16),
        # prefill of four prompts, from slices of fused projections
        scan("scan_prefill_bf16", "fwd", "bf16", 4, 4096, 4096, 16, fused=True),
        # an ordinary training step
        scan("scan_train_bf16", "train", "bf16", 8, 2048, 2048, 16),
        # packed documents, two groups of channels with B and C of their own
        scan("scan_packed_f16_train", "train", "f16", 60, 30_011, 1000, 16, groups=2, packed=True,
             h0=True),
        # one long sequence of few channels and states in full precision, ungated
        scan("scan_long_f32_train", "train", "f32", 1, 65_536, 512, 8, h0=True, z=False),
        # before a block in serving: 16 tokens
        norm("norm_in_step_bf16", "in", "fwd", "bf16", "bf16", 16, 4096),
        # before a block in training, the residual stream in 32 bits
        norm("norm_in_train_bf16", "in", "train", "bf16", "f32", 16_384, 2048, scale=True),
        # after a block in training: the gate is half of a fused projection
        norm("norm_out_train_bf16", "out", "train", "bf16", "bf16", 16_384, 4096, fused=True),
        # after a block, an odd width, gate behind the norm, scaled onto the residual
        norm("norm_out_odd_f32_train", "out", "train", "f32", "f32", 5003, 1001, order="norm_first",
             scale=True, residual=True),
    ]


def conv(name, do, dtype, seqs, steps, dim, width, act="silu", state=False, fused=False,
         packed=False):
    c = {"op": "conv", "do": do, "dtype": dtype, "seqs": seqs, "steps": steps, "dim": dim,
         "width": width, "act": act, "state": state or do == "step", "fused": fused,
         "packed": packed}
    return dict(c, name=name) if name else c


def scan(name, do, dtype, seqs, steps, dim, states, groups=1, z=True, h0=False, fused=False,
         packed=False):
    c = {"op": "scan", "do": do, "dtype": dtype, "seqs": seqs, "steps": steps, "dim": dim,
         "states": states, "groups": groups, "z": z, "h0": h0 or do == "step", "fused": fused,
         "packed": packed}
    return dict(c, name=name) if name else c


def norm(name, side, do, dtype, stream, rows, dim, order="gate_first", scale=False, residual=None,
         fused=False):
    """`stream`: the residual's type."""
    residual = (side == "in") if residual is None else residual
    c = {"op": "norm_" + side, "do": do, "dtype": dtype, "stream": stream, "rows": rows, "dim": dim,
         "order": order, "scale": scale, "residual": residual, "fused": fused}
    return dict(c, name=name) if name else c


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def channels(rng, lo, hi):
    d = log_int(rng, lo, hi)
    return max(8, d // 8 * 8) if rng.random() < 0.7 else d


def draw(rng):
    kind = rng.choice(["conv", "scan", "scan", "norm"])
    dtype = rng.choice(list(DTYPES))
    if kind == "norm":
        do = rng.choice(["fwd", "train"])
        dim = channels(rng, 32, 16_384)
        rows = log_int(rng, 1, min(100_000, 67_108_864 // dim))
        stream = "f32" if rng.random() < 0.3 else dtype
        if rng.random() < 0.5:
            residual = rng.random() < 0.8
            return norm(None, "in", do, dtype, stream if residual else dtype, rows, dim,
                        scale=residual and rng.random() < 0.5, residual=residual)
        residual = rng.random() < 0.5
        return norm(None, "out", do, dtype, stream if residual else dtype, rows, dim,
                    order=rng.choice(["gate_first", "norm_first"]), scale=rng.random() < 0.5,
                    residual=residual, fused=rng.random() < 0.4)
    do = rng.choice(["step", "fwd", "train", "train"])
    dim = channels(rng, 16, 8192)
    if do == "step":
        seqs = log_int(rng, 1, 256)
        if kind == "conv":
            return conv(None, do, dtype, seqs, 1, dim, rng.randint(2, 4),
                        rng.choice(["silu", "none"]))
        return scan(None, do, dtype, seqs, 1, dim, rng.randint(1, 16), z=rng.random() < 0.7)
    packed = rng.random() < 0.35
    if kind == "conv":
        elems = 67_108_864 if do == "fwd" else 33_554_432
        states = 1
    else:
        states = rng.choice([16, 16, 8, 4, rng.randint(1, 16)])
        elems = (1_073_741_824 if do == "fwd" else 402_653_184) // max(states, 4)
    steps = log_int(rng, 1, min(100_000, elems // dim))
    seqs = log_int(rng, 1, min(256, steps if packed else elems // dim // steps))
    fused, first = rng.random() < 0.3, rng.random() < 0.5
    if kind == "conv":
        return conv(None, do, dtype, seqs, steps, dim, rng.randint(2, 4),
                    rng.choice(["silu", "silu", "none"]), first, fused, packed)
    groups = 2 if dim % 2 == 0 and rng.random() < 0.25 else 1
    return scan(None, do, dtype, seqs, steps, dim, states, groups, rng.random() < 0.7, first, fused,
                packed)


# ----- inputs -----

def lengths(case, seed):
    """Packed sequences' lengths: from empty to many times the mean."""
    r = np.random.RandomState(seed % (1 << 31))
    w = r.exponential(1.0, case["seqs"]) ** 2
    if case["seqs"] > 3:
        w[1] = 0.0
    n = np.floor(w / w.sum() * case["steps"]).astype(np.int64)
    if case["seqs"] > 3:
        n[2] = 1
    n[int(np.argmax(n))] += case["steps"] - n.sum()
    return n


def randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g, dtype=torch.float32)


def halves(g, case, lead, *sizes):
    """Normal tensors (lead, size): slices of one wide tensor where the case says so."""
    dt = DTYPES[case["dtype"]]
    if not case["fused"]:
        return [randn(g, *lead, n).to(dt) for n in sizes]
    return list(randn(g, *lead, sum(sizes)).to(dt).split(sizes, -1))


def seq_inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    lead = (case["steps"],) if case["packed"] else (case["seqs"], case["steps"])
    s = {"case": case, "offsets": None}
    if case["packed"]:
        n = lengths(case, seed)
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to(DEV)
        s["longest"] = int(n.max())
    return g, lead, s


def conv_inputs(case, seed):
    """Weights of the usual first size, 1 / sqrt(width)."""
    g, lead, s = seq_inputs(case, seed)
    d, k, dt = case["dim"], case["width"], DTYPES[case["dtype"]]
    s["x"], s["other"] = halves(g, case, lead, d, d if case["fused"] else 0)
    s["weight"] = (torch.rand(d, k, device=DEV, generator=g) * 2 - 1) / math.sqrt(k)
    s["bias"] = (torch.rand(d, device=DEV, generator=g) * 2 - 1) / math.sqrt(k)
    s["state"] = randn(g, case["seqs"], k - 1, d).to(dt) if case["state"] else None
    if case["do"] == "train":
        s["dy"] = randn(g, *lead, d).to(dt)
        s["dlast"] = randn(g, case["seqs"], k - 1, d).to(dt)
    return s


def scan_inputs(case, seed):
    """Steps from 0.001 to 0.1 at rest, decay rates about 1 .. N, as models are begun."""
    g, lead, s = seq_inputs(case, seed)
    d, n, gr = case["dim"], case["states"], case["groups"]
    s["x"], s["z"] = halves(g, case, lead, d, d)
    if not case["z"]:
        s["z"] = None
    s["dt"], b, c = halves(g, case, lead, d, gr * n, gr * n)
    s["B"], s["C"] = b.unflatten(-1, (gr, n)), c.unflatten(-1, (gr, n))
    rate = torch.arange(1, n + 1, device=DEV, dtype=torch.float32)
    s["A"] = -rate * (0.3 * randn(g, d, n)).exp()
    s["D"] = 1 + 0.1 * randn(g, d)
    rest = torch.exp(torch.rand(d, device=DEV, generator=g) * math.log(100.0) + math.log(1e-3))
    s["bias"] = torch.log(torch.expm1(rest))
    s["h0"] = 0.3 * randn(g, case["seqs"], d, n) if case["h0"] else None
    if case["do"] == "train":
        s["dy"] = randn(g, *lead, d).to(DTYPES[case["dtype"]])
        s["dlast"] = randn(g, case["seqs"], d, n)
    return s


def norm_inputs(case, seed):
    """A residual stream a few times as large as what a block adds to it."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, d = case["rows"], case["dim"]
    dt, rt = DTYPES[case["dtype"]], DTYPES[case["stream"]]
    s = {"case": case, "gate": None, "residual": None, "scale": None}
    if case["op"] == "norm_out":
        s["x"], s["gate"] = halves(g, case, (rows,), d, d)
    else:
        s["x"] = randn(g, rows, d).to(dt)
    s["weight"] = 1 + 0.2 * randn(g, d)
    if case["residual"]:
        s["residual"] = (3 * randn(g, rows, d)).to(rt)
    if case["scale"]:
        s["scale"] = 0.5 + 0.2 * randn(g, d)
    if case["do"] == "train":
        s["dy"] = randn(g, rows, d).to(dt if case["op"] == "norm_in" else rt)
        if case["op"] == "norm_in" and case["residual"]:
            s["dr"] = randn(g, rows, d).to(rt)
    return s


INPUTS = {"conv": conv_inputs, "scan": scan_inputs, "norm_in": norm_inputs, "norm_out": norm_inputs}


def prepare(case, seed):
    return INPUTS[case["op"]](case, seed)


# ----- one pass -----

def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


def conv_own(s):
    from preconditioned_cg_solver_amd import binding as B
    c = s["case"]
    if c["do"] == "step":  # the state is updated in place
        y, last = B.sla_conv_forward(s["x"], s["weight"], bias=s["bias"], state=s["state"],
                                     act=c["act"], last=s["state"])
        return {"y": y, "last": last}
    y, last = B.sla_conv_forward(s["x"], s["weight"], bias=s["bias"], state=s["state"],
                                 offsets=s["offsets"], act=c["act"])
    out = {"y": y, "last": last}
    if c["do"] == "train":
        out["dx"], out["dw"], out["db"], out["dstate"] = B.sla_conv_backward(
            s["x"], s["weight"], s["dy"], bias=s["bias"], state=s["state"], grad_last=s["dlast"],
            offsets=s["offsets"], act=c["act"])
    return out


def scan_own(s):
    from preconditioned_cg_solver_amd import binding as B
    c = s["case"]
    common = dict(D=s["D"], z=s["z"], dt_bias=s["bias"], h0=s["h0"], offsets=s["offsets"],
                  softplus=True)
    first = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    if c["do"] == "step":
        y, last, _ = B.sla_selscan_forward(*first, **common, h_last=s["h0"])
        return {"y": y, "last": last}
    train = c["do"] == "train"
    y, last, saved = B.sla_selscan_forward(*first, **common, save=train)
    out = {"y": y, "last": last}
    if train:
        names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")
        out.update(zip(names, B.sla_selscan_backward(*first, saved, s["dy"], grad_last=s["dlast"],
                                                     **common)))
    return out


def norm_own(s):
    from preconditioned_cg_solver_amd import binding as B
    c = s["case"]
    if c["op"] == "norm_in":
        y, r, rstd = B.sla_norm_in_forward(s["x"], s["weight"], residual=s["residual"],
                                           scale=s["scale"], eps=EPS)
        out = {"y": y, "r": r}
        if c["do"] == "train":
            out["dx"], dres, out["dw"], out["dscale"] = B.sla_norm_in_backward(
                s["dy"], s["x"], s["weight"], rstd, residual=s["residual"], scale=s["scale"],
                grad_r=s.get("dr"))
            out["dres"] = dres if c["residual"] else None
        return out
    y, rstd = B.sla_norm_out_forward(s["x"], s["weight"], gate=s["gate"], residual=s["residual"],
                                     scale=s["scale"], order=c["order"], eps=EPS)
    out = {"y": y}
    if c["do"] == "train":
        out["dx"], out["dgate"], out["dw"], out["dscale"] = B.sla_norm_out_backward(
            s["dy"], s["x"], s["weight"], rstd, gate=s["gate"], scale=s["scale"], order=c["order"])
    return out


def bounds(s):
    """Packed sequences that are not empty: which, their first and last steps."""
    off = s["offsets"]
    some = off[1:] > off[:-1]
    return some, off[:-1][some], off[1:][some] - 1


def silu(v):
    sg = torch.sigmoid(v)
    return v * sg, sg * (1 + v * (1 - sg))


def conv_parts(s, dt):
    """x, and the inputs that stand before each sequence, in type dt."""
    c = s["case"]
    x = s["x"].to(dt)
    state = s["state"].to(dt) if s["state"] is not None else \
        x.new_zeros(c["seqs"], c["width"] - 1, c["dim"])
    return x, state


def conv_plain(s):
    c, k, dt = s["case"], s["case"]["width"], DTYPES[s["case"]["dtype"]]
    x, state = conv_parts(s, torch.float32)
    w, steps = s["weight"], c["steps"]
    n = c["seqs"]
    if c["packed"]:  # every sequence behind its state, in one long row
        off = s["offsets"]
        of = torch.searchsorted(off, torch.arange(steps, device=DEV), right=True) - 1
        at = torch.arange(steps, device=DEV) + (of + 1) * (k - 1)  # where a step lies in the row
        row = x.new_zeros(steps + n * (k - 1), c["dim"])
        head = (off[:-1] + torch.arange(n, device=DEV) * (k - 1))[:, None] + \
            torch.arange(k - 1, device=DEV)
        row[head] = state
        row[at] = x
        tail = (off[1:] + torch.arange(1, n + 1, device=DEV) * (k - 1))[:, None] - k + 1 + \
            torch.arange(k - 1, device=DEV)
        last = row[tail]
        pre = s["bias"] + sum(w[:, j] * row[at - k + 1 + j] for j in range(k))
    else:
        row = torch.cat([state, x], 1)
        last = row[:, steps:]
        pre = s["bias"] + sum(w[:, j] * row[:, j:j + steps] for j in range(k))
    y, slope = silu(pre) if c["act"] == "silu" else (pre, torch.ones_like(pre))
    out = {"y": y.to(dt), "last": last.to(dt)}
    if c["do"] == "step":
        s["state"].copy_(last)
        out["last"] = s["state"]
    if c["do"] != "train":
        return out
    dpre = s["dy"].float() * slope
    drow, dlast = torch.zeros_like(row), s["dlast"].float()
    dw = torch.empty_like(w)
    flat = dpre.reshape(-1, c["dim"])
    for j in range(k):
        if c["packed"]:
            drow.index_add_(0, at - k + 1 + j, w[:, j] * dpre)
            dw[:, j] = (flat * row[at - k + 1 + j]).sum(0)
        else:
            drow[:, j:j + steps] += w[:, j] * dpre
            dw[:, j] = (flat * row[:, j:j + steps].reshape(-1, c["dim"])).sum(0)
    if c["packed"]:
        drow.index_add_(0, tail.flatten(), dlast.flatten(0, 1))
        dx, dstate = drow[at], drow[head]
    else:
        drow[:, steps:] += dlast
        dx, dstate = drow[:, k - 1:], drow[:, :k - 1]
    return dict(out, dx=dx.to(dt), dw=dw, db=flat.sum(0),
                dstate=dstate.to(dt) if c["state"] else None)


def doubling(a, b, longest):
    """b_t + a_t b_{t-1} + a_t a_{t-1} b_{t-2} + ... along dimension 1."""
    k = 1
    while k < longest:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def scan_plain(s):
    c, dt_ = s["case"], DTYPES[s["case"]["dtype"]]
    packed, train, d = c["packed"], c["do"] == "train", c["dim"]

    def load(t):
        return t.float().unsqueeze(0) if packed else t.float()

    def back(t):
        return t[0] if packed else t

    x, u, z = load(s["x"]), load(s["dt"]) + s["bias"], None
    delta = u.clamp(min=0) + torch.log1p(torch.exp(-u.abs()))
    bx, cx = load(s["B"]), load(s["C"])
    if s["z"] is not None:
        z, zslope = silu(load(s["z"]))
    h0 = s["h0"] if s["h0"] is not None else x.new_zeros(c["seqs"], d, c["states"])
    last = h0.clone()
    if packed:
        some, first, end = bounds(s)
        longest = s["longest"]
    else:
        longest = c["steps"]
    sums, dx, ddelta = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    da, dh0 = torch.empty_like(s["A"]), torch.empty_like(h0)
    db, dc = torch.empty_like(bx), torch.empty_like(cx)
    wide = [t.repeat_interleave(d // c["groups"], 2) if c["groups"] > 1 else t for t in (bx, cx)]
    kept = []
    for n in range(c["states"]):  # the states are independent until they are summed
        a = torch.exp(delta * s["A"][:, n])
        b, across = delta * x * wide[0][..., n], a.clone()
        if packed:
            b[0, first] += a[0, first] * h0[some][..., n]
            across[0, first] = 0
        else:
            b[:, 0] += a[:, 0] * h0[..., n]
            across[:, 0] = 0
        h = doubling(across, b, longest)
        if packed:
            last[some, :, n] = h[0, end]
        else:
            last[..., n] = h[:, -1]
        sums += wide[1][..., n] * h
        if train:
            kept.append((a, across, h))
    sums += s["D"] * x
    out = {"y": back(sums if z is None else sums * z).to(dt_), "last": last}
    if c["do"] == "step":
        s["h0"].copy_(last)
        out["last"] = s["h0"]
    if not train:
        return out
    dy = load(s["dy"])
    ds = dy if z is None else dy * z
    for n, (a, across, h) in enumerate(kept):
        b = ds * wide[1][..., n]
        before = torch.cat([h[:, :1], h[:, :-1]], 1)
        if packed:
            b[0, end] += s["dlast"][some][..., n]
            before[0, first] = h0[some][..., n]
        else:
            b[:, -1] += s["dlast"][..., n]
            before[:, 0] = h0[..., n]
        into = torch.cat([across[:, 1:], torch.zeros_like(across[:, :1])], 1)
        g = doubling(into.flip(1), b.flip(1), longest).flip(1)
        q = g * a * before
        da[:, n] = (q * delta).sum((0, 1))
        ddelta += q * s["A"][:, n] + g * x * wide[0][..., n]
        dx += g * wide[0][..., n]
        by = (c["groups"], d // c["groups"])
        db[..., n] = (g * delta * x).unflatten(2, by).sum(3)
        dc[..., n] = (ds * h).unflatten(2, by).sum(3)
        dh0[..., n] = s["dlast"][..., n]
        if packed:
            dh0[some, :, n] = a[0, first] * g[0, first]
        else:
            dh0[..., n] = a[:, 0] * g[:, 0]
    du = ddelta * torch.sigmoid(u)
    return dict(out, dx=back(delta * dx + s["D"] * ds).to(dt_), ddt=back(du).to(dt_), dA=da,
                dB=back(db).to(dt_), dC=back(dc).to(dt_), dD=(ds * x).sum((0, 1)),
                dz=None if z is None else back(dy * sums * zslope).to(dt_),
                dbias=du.sum((0, 1)), dh0=dh0 if c["h0"] else None)


def norm_plain(s):
    c, dt, rt = s["case"], DTYPES[s["case"]["dtype"]], DTYPES[s["case"]["stream"]]
    x, w, scale = s["x"].float(), s["weight"], s["scale"]
    res = s["residual"].float() if s["residual"] is not None else None
    train = c["do"] == "train"
    if c["op"] == "norm_in":
        r = x if scale is None else x * scale
        r = r if res is None else res + r
        rstd = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
        out = {"y": (r * rstd * w).to(dt), "r": r.to(rt)}
        if not train:
            return out
        dy = s["dy"].float()
        hat, g = r * rstd, dy * w
        dr = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
        if res is not None:
            dr = dr + s["dr"].float()
        return dict(out, dx=(dr if scale is None else dr * scale).to(dt),
                    dres=dr.to(rt) if res is not None else None, dw=(dy * hat).sum(0),
                    dscale=None if scale is None else (dr * x).sum(0))
    gate, slope = silu(s["gate"].float())
    u = x * gate if c["order"] == "gate_first" else x
    rstd = torch.rsqrt(u.square().mean(1, keepdim=True) + EPS)
    hat = u * rstd
    n = hat * w if c["order"] == "gate_first" else hat * w * gate
    y = n if scale is None else n * scale
    out = {"y": (y if res is None else res + y).to(rt)}
    if not train:
        return out
    dy = s["dy"].float()
    dn = dy if scale is None else dy * scale
    dhat = dn * w if c["order"] == "gate_first" else dn * w * gate
    du = rstd * (dhat - hat * (dhat * hat).mean(1, keepdim=True))
    if c["order"] == "gate_first":
        dx, dgate, dw = du * gate, du * x * slope, dn * hat
    else:
        dx, dgate, dw = du, dn * hat * w * slope, dn * hat * gate
    return dict(out, dx=dx.to(dt), dgate=dgate.to(dt), dw=dw.sum(0),
                dscale=None if scale is None else (dy * n).sum(0))


OWN = {"conv": conv_own, "scan": scan_own, "norm_in": norm_own, "norm_out": norm_own}
PLAIN = {"conv": conv_plain, "scan": scan_plain, "norm_in": norm_plain, "norm_out": norm_plain}


# ----- work -----

def work(case):
    e, d = BYTES[case["dtype"]], case["dim"]
    train = case["do"] == "train"
    if case["op"].startswith("norm"):
        n, r = case["rows"] * d, BYTES[case["stream"]]
        if case["op"] == "norm_in":  # x, residual; y, r (r is x where there is no residual)
            each = 2 * e + (2 * r if case["residual"] else 0)
            if train:  # dy, dr; dx, dresidual
                each += 2 * e + (2 * r if case["residual"] else 0)
            return {"bytes": each * n + 4 * d, "flops": (20 if train else 6) * n}
        each = 2 * e + r * (2 if case["residual"] else 1)
        if train:  # dout; dx, dgate
            each += r + 2 * e
        return {"bytes": each * n + 4 * d, "flops": (40 if train else 14) * n}
    tokens = case["steps"] if case["packed"] else case["seqs"] * case["steps"]
    n = tokens * d
    if case["op"] == "conv":
        k = case["width"]
        held = e * case["seqs"] * (k - 1) * d  # states
        if not train:
            return {"bytes": 2 * e * n + held * (2 if case["state"] else 1) + 4 * (k + 1) * d,
                    "flops": (2 * k + 6) * n}
        return {"bytes": 4 * e * n + held * (4 if case["state"] else 2) + 8 * (k + 1) * d,
                "flops": (6 * k + 20) * n}
    k, z = case["states"], 1 if case["z"] else 0
    held = 4 * case["seqs"] * d * k
    shared = 2 * e * tokens * case["groups"] * k
    if not train:
        return {"bytes": (3 + z) * e * n + shared + held * (2 if case["h0"] else 1) + 4 * d * (k + 2),
                "flops": (7 * k + 20) * n}
    # x, dt, z, dy in; y, dx, ddt, dz out; B, C and their gradients; the states and theirs
    return {"bytes": (6 + 2 * z) * e * n + 2 * shared + held * (4 if case["h0"] else 2)
            + 8 * d * (k + 2), "flops": (24 * k + 60) * n}


# ----- 64 bits -----

def exact(case, seed):
    s = INPUTS[case["op"]](case, seed)
    return {"conv": conv_exact, "scan": scan_exact}.get(case["op"], norm_exact)(s)


def conv_exact(s):
    """Sequence by sequence; the gradients by torch's differentiation of the sum."""
    c, k = s["case"], s["case"]["width"]
    w, b = s["weight"].double().requires_grad_(), s["bias"].double().requires_grad_()
    x, state = conv_parts(s, torch.float64)
    x.requires_grad_(), state.requires_grad_()
    off = s["offsets"].tolist() if c["packed"] else None
    parts = [(x[a:e], state[i]) for i, (a, e) in enumerate(zip(off, off[1:]))] if c["packed"] \
        else [(x.transpose(0, 1), state.transpose(0, 1))]
    ys, lasts = [], []
    for seq, head in parts:
        row = torch.cat([head, seq])
        pre = b.clone()
        for j in range(k):
            pre = pre + row[j:len(row) - k + 1 + j] * w[:, j]
        ys.append(pre / (1 + (-pre).exp()) if c["act"] == "silu" else pre)
        lasts.append(row[len(row) - k + 1:])
    y = torch.cat(ys) if c["packed"] else ys[0].transpose(0, 1)
    last = torch.stack(lasts) if c["packed"] else lasts[0].transpose(0, 1)
    out = {"y": y.detach(), "last": last.detach()}
    if c["do"] == "train":
        got = torch.autograd.grad([y, last], [x, w, b, state],
                                  [s["dy"].double(), s["dlast"].double()])
        out.update(dx=got[0], dw=got[1], db=got[2], dstate=got[3] if c["state"] else None)
    return out


def scan_exact(s):
    """Step by step in 64 bits, time first; packed sequences as one, cut where each begins."""
    c, d, k = s["case"], s["case"]["dim"], s["case"]["states"]
    T, per = c["steps"], d // c["groups"]
    turn = (lambda t: t.double()) if c["packed"] else (lambda t: t.double().transpose(0, 1))
    x, u = turn(s["x"]), turn(s["dt"]) + s["bias"].double()
    delta = torch.where(u > 30, u, (u.clamp(max=30).exp() + 1).log())
    delta = torch.where(u < -30, u.exp(), delta)
    B, C = (turn(s[v]).repeat_interleave(per, -2) for v in "BC")
    A, D = s["A"].double(), s["D"].double()
    a = (delta.unsqueeze(-1) * A).exp_()
    h = (delta * x).unsqueeze(-1) * B
    h0 = s["h0"].double() if s["h0"] is not None else x.new_zeros(c["seqs"], d, k)
    if c["packed"]:
        off = s["offsets"].tolist()
        live = [i for i in range(c["seqs"]) if off[i + 1] > off[i]]
        first = torch.tensor([off[i] for i in live], device=DEV)
        end = torch.tensor([off[i + 1] - 1 for i in live], device=DEV)
        of = torch.tensor(live, device=DEV)
        starts, ends = set(first.tolist()), set(end.tolist())
    else:
        first, end, of, starts, ends = 0, T - 1, slice(None), {0}, {T - 1}
    h[first] += a[first] * h0[of]
    for t in range(1, T):
        if t not in starts:
            h[t].addcmul_(a[t], h[t - 1])
    last = h0.clone()
    last[of] = h[end]
    total = (h * C).sum(-1) + D * x
    z = turn(s["z"]) if s["z"] is not None else None
    gate = z / (1 + (-z).exp()) if z is not None else 1.0
    out = {"y": turn(total * gate), "last": last}
    if c["do"] != "train":
        return out
    dy = turn(s["dy"])
    ds = dy * gate
    g = ds.unsqueeze(-1) * C
    g[end] += s["dlast"].double()[of]
    for t in range(T - 2, -1, -1):
        if t not in ends:
            g[t].addcmul_(a[t + 1], g[t + 1])
    out["dh0"] = None
    if s["h0"] is not None:
        out["dh0"] = s["dlast"].double()
        out["dh0"][of] = a[first] * g[first]
    across = tuple(range(x.dim() - 1))
    by = (c["groups"], per)
    out["dB"] = turn(((delta * x).unsqueeze(-1) * g).unflatten(-2, by).sum(-2))
    out["dC"] = turn((ds.unsqueeze(-1) * h).unflatten(-2, by).sum(-2))
    del C
    gb = (g * B).sum(-1)
    del B
    before = torch.cat([h[:1], h[:-1]])
    del h
    before[first] = h0[of]
    q = before.mul_(a).mul_(g)
    del a, g
    out["dA"] = (q * delta.unsqueeze(-1)).sum(across)
    du = ((q * A).sum(-1) + x * gb) / (1 + (-u).exp())
    out["dz"] = None
    if z is not None:
        sg = 1 / (1 + (-z).exp())
        out["dz"] = turn(dy * total * (sg + z * sg * (1 - sg)))
    out.update(dx=turn(delta * gb + D * ds), ddt=turn(du), dD=(ds * x).sum(across),
               dbias=du.sum(across))
    return out


def norm_exact(s):
    """By torch's differentiation of the definition."""
    c = s["case"]
    names = ("x", "weight", "gate", "residual", "scale")
    v = {n: s[n].double().requires_grad_() if s[n] is not None else None for n in names}
    scale = v["scale"] if v["scale"] is not None else 1.0
    res = v["residual"] if v["residual"] is not None else 0.0

    def over(t):
        return t / ((t * t).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt() * v["weight"]

    if c["op"] == "norm_in":
        r = res + scale * v["x"]
        out, grads = {"y": over(r), "r": r}, {"y": "dy", "r": "dr"}
        want = {"dx": "x", "dres": "residual", "dw": "weight", "dscale": "scale"}
    else:
        gate = v["gate"] / (1 + (-v["gate"]).exp())
        n = over(v["x"] * gate) if c["order"] == "gate_first" else over(v["x"]) * gate
        out, grads = {"y": res + scale * n}, {"y": "dy"}
        want = {"dx": "x", "dgate": "gate", "dw": "weight", "dscale": "scale"}
    got = {}
    if c["do"] == "train":
        ends = [k for k in grads if s.get(grads[k]) is not None]
        leaves = [v[n] for n in want.values() if v[n] is not None]
        back = iter(torch.autograd.grad([out[k] for k in ends], leaves,
                                        [s[grads[k]].double() for k in ends]))
        got = {k: next(back) if v[n] is not None else None for k, n in want.items()}
    return dict({k: t.detach() for k, t in out.items()}, **got)

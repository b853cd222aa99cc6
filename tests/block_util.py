"""Plain references, in 64 bits, of the operators of a sequence block (causal
convolution, selective scan, norms) and their gradients, with running bounds on how
far a computation in fewer bits may be off (numpy, no library code).

A Num is a value and a bound on its error in unit roundoff u: a sum or product adds u
times its size to what its operands bring, an elementary function 4 u (the
hardware's exponential, logarithm, reciprocal and root are within one unit in the last
place, 2 u) and what its argument's error makes of it, a sum of n terms in any order
(n - 1) u times the sum of their sizes.  Where the operators associate differently than
written here the rounding counts are the same to first order; `slack` covers the
second, and joins of a recurrence's parts."""
from __future__ import annotations

import numpy as np

U32, U64 = 2.0 ** -24, 2.0 ** -53
# half the spacing of the storage types, relative; and half their smallest step
STORE = {"f64": (2.0 ** -53, 2.0 ** -1074), "f32": (2.0 ** -24, 2.0 ** -149),
         "bf16": (2.0 ** -8, 2.0 ** -133), "f16": (2.0 ** -11, 2.0 ** -25)}
SLACK = 1.5


class Num:
    __array_ufunc__ = None  # an array times a Num is a Num

    def __init__(self, v, e=0.0, u=U32):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(e, dtype=np.float64), self.v.shape)
        self.u = u

    def _of(self, o):
        return o if isinstance(o, Num) else Num(o, 0.0, self.u)

    def _made(self, v, e):
        return Num(v, e + self.u * np.abs(v), self.u)

    def __add__(self, o):
        o = self._of(o)
        return self._made(self.v + o.v, self.e + o.e)

    __radd__ = __add__

    def __neg__(self):
        return Num(-self.v, self.e, self.u)

    def __sub__(self, o):
        return self + (-self._of(o))

    def __rsub__(self, o):
        return self._of(o) + (-self)

    def __mul__(self, o):
        o = self._of(o)
        return self._made(self.v * o.v,
                          np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e)

    __rmul__ = __mul__

    def __getitem__(self, k):
        return Num(self.v[k], self.e[k], self.u)

    def fn(self, f, slope):
        """f of it, the derivative's size at most `slope` nearby."""
        v = f(self.v)
        return Num(v, 4 * self.u * np.abs(v) + slope * self.e, self.u)

    def sum(self, axis):
        n = np.prod([self.v.shape[a] for a in np.atleast_1d(axis)])
        axis = tuple(np.atleast_1d(axis))
        return Num(self.v.sum(axis), (self.e + n * self.u * np.abs(self.v)).sum(axis), self.u)

    def stored(self, to):
        """(value, bound) once rounded to a storage type."""
        r, tiny = STORE[to]
        # in fp64 the reference is off by as much itself
        e = SLACK * (2 if self.u == U64 else 1) * self.e
        return self.v, e + r * (np.abs(self.v) + e) + tiny


def stack(parts, axis=0):
    return Num(np.stack([p.v for p in parts], axis), np.stack([p.e for p in parts], axis),
               parts[0].u)


def zeros(shape, u):
    return Num(np.zeros(shape), 0.0, u)


def sigmoid64(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def sigmoid(x):
    # relative error of e^-v is the rounding of the argument, |v| u, and 4 u
    s = sigmoid64(x.v)
    return Num(s, (8 + np.abs(x.v)) * x.u * s + x.e / 4, x.u)


def silu(x):
    return x * sigmoid(x)


def silu_slope(x):
    s = sigmoid(x)
    return s + x * (s * (1.0 - s))


def softplus(x):
    v = np.maximum(x.v, 0) + np.log1p(np.exp(-np.abs(x.v)))
    s = sigmoid64(x.v)
    # log(1 + e): e is off by (|v| + 4) u, relative, which e / (1 + e) damps
    return Num(v, x.u * (8 * np.abs(v) + (np.abs(x.v) + 8) * s) + s * x.e, x.u)


def exp(x):
    v = np.exp(x.v)
    # the argument is scaled to a power of two and rounded twice
    return Num(v, v * (x.u * (6 + 3 * np.abs(x.v)) + x.e), x.u)


def spans(lead, offsets):
    """Index of each sequence in arrays of leading shape `lead`."""
    if offsets is None:
        return [(s, slice(None)) for s in range(lead[0])]
    return [(slice(int(a), int(b)),) for a, b in zip(offsets[:-1], offsets[1:])]


# ----- causal convolution -----

def conv(x, w, bias, state, offsets, act, dy=None, dlast=None, unit=U32, store="f32"):
    """{name: (value, bound)} of every output."""
    k, d = w.shape[1], w.shape[0]
    own = "f64" if unit == U64 else "f32"
    n = (len(offsets) - 1) if offsets is not None else x.shape[0]
    W = Num(w, 0, unit)
    b = Num(bias if bias is not None else np.zeros(d), 0, unit)
    y, ye = np.zeros_like(x), np.zeros_like(x)
    dx, dxe = np.zeros_like(x), np.zeros_like(x)
    last = np.zeros((n, k - 1, d))
    dst, dste = np.zeros((n, k - 1, d)), np.zeros((n, k - 1, d))
    dw, db = [], []
    for s, at in enumerate(spans(x.shape, offsets)):
        head = np.zeros((k - 1, d)) if state is None else state[s]
        row = np.concatenate([head, x[at]])
        t = len(row) - k + 1
        last[s] = row[t:]
        pre = b + zeros((t, d), unit)
        for j in range(k):
            pre = pre + W[:, j] * row[j:j + t]
        out = silu(pre) if act == "silu" else pre
        y[at], ye[at] = out.stored(store)
        if dy is None:
            continue
        g = Num(dy[at], 0, unit) * (silu_slope(pre) if act == "silu" else 1.0)
        drow = [zeros((d,), unit) for _ in range(len(row))]
        for i in range(t):
            for j in range(k):
                drow[i + j] = drow[i + j] + W[:, j] * g[i]
        for j in range(k - 1):
            drow[t + j] = drow[t + j] + (dlast[s, j] if dlast is not None else 0.0)
        if len(drow):
            all_ = stack(drow)
            v, e = all_.stored(store)
            dx[at], dxe[at] = v[k - 1:], e[k - 1:]
            dst[s], dste[s] = v[:k - 1], e[:k - 1]
        dw.append([g * row[j:j + t] for j in range(k)])
        db.append(g)
    out = {"y": (y, ye), "last": (last, np.zeros_like(last))}
    if dy is None:
        return out
    out["dx"], out["dstate"] = (dx, dxe), (dst, dste)

    def total(parts):
        v = np.concatenate([p.v for p in parts]) if parts else np.zeros((0, d))
        e = np.concatenate([p.e for p in parts]) if parts else np.zeros((0, d))
        return Num(v, e, unit).sum(0)

    cols = [total([p[j] for p in dw]) for j in range(k)]
    out["dw"] = stack(cols, 1).stored(own)
    out["db"] = total(db).stored(own)
    return out


# ----- selective scan -----

def scan(x, dt, A, B, C, D=None, z=None, bias=None, h0=None, offsets=None, softplus_=True, dy=None,
         dlast=None, unit=U32, store="f32"):
    """{name: (value, bound)} of every output; B and C (.., groups, states)."""
    own = "f64" if unit == U64 else "f32"
    d, N = A.shape
    per = d // B.shape[-2]
    n = (len(offsets) - 1) if offsets is not None else x.shape[0]
    An = Num(A, 0, unit)
    Dn = Num(D if D is not None else np.zeros(d), 0, unit)
    names = ["y"] + (["dx", "ddt", "dz"] if dy is not None else [])
    outs = {k: (np.zeros_like(x), np.zeros_like(x)) for k in names}
    shared = {k: (np.zeros_like(B), np.zeros_like(B)) for k in ("dB", "dC")}
    last, laste = np.zeros((n, d, N)), np.zeros((n, d, N))
    dh0, dh0e = np.zeros((n, d, N)), np.zeros((n, d, N))
    sums = {"dA": [], "dD": [], "dbias": []}
    for s, at in enumerate(spans(x.shape, offsets)):
        xs, T = x[at], x[at].shape[0]
        u = Num(dt[at], 0, unit) + (bias if bias is not None else 0.0)
        delta = softplus(u) if softplus_ else u
        wide = [np.repeat(t[at], per, axis=-2) for t in (B, C)]  # (T, d, N)
        arg = delta[..., None] * An
        a = exp(arg)
        # joins: a chunk's coefficients are one exponential of the sum of its deltas, which
        # is off by a rounding for each of its tiles, and carried on by 4 factors
        a = Num(a.v, a.e + unit * a.v * (6 + np.abs(arg.v) * (8 + T / 8)), unit)
        into = (delta * xs)[..., None] * wide[0]
        state = Num(h0[s] if h0 is not None else np.zeros((d, N)), 0, unit)
        first, hs = state, []
        for t in range(T):
            state = a[t] * state + into[t]
            hs.append(state)
        last[s], laste[s] = state.stored(own)
        if T == 0:
            dh0[s] = dlast[s] if dlast is not None else 0.0
            continue
        h = stack(hs)
        total = (h * wide[1]).sum(2) + Dn * xs
        gate = silu(Num(z[at], 0, unit)) if z is not None else 1.0
        outs["y"][0][at], outs["y"][1][at] = (total * gate).stored(store)
        if dy is None:
            continue
        g_y = Num(dy[at], 0, unit)
        ds = g_y * gate
        if z is not None:
            dz = g_y * total * silu_slope(Num(z[at], 0, unit))
            outs["dz"][0][at], outs["dz"][1][at] = dz.stored(store)
        mu = Num(dlast[s] if dlast is not None else np.zeros((d, N)), 0, unit)
        gs, mus = [None] * T, [None] * T
        for t in range(T - 1, -1, -1):
            gs[t] = ds[t][:, None] * wide[1][t] + mu
            mu = a[t] * gs[t]
            mus[t] = mu
        dh0[s], dh0e[s] = mu.stored(own)
        g, m = stack(gs), stack(mus)
        q = m * stack([first] + hs[:-1])
        gb = (g * wide[0]).sum(2)
        # the kernels sum over n before they multiply by A in powers of two: 2 more
        du = (q * An).sum(2) + xs * gb
        du = Num(du.v, du.e + 4 * unit * np.abs(du.v), unit)
        if softplus_:
            du = du * sigmoid(u)
        outs["dx"][0][at], outs["dx"][1][at] = (delta * gb + Dn * ds).stored(store)
        outs["ddt"][0][at], outs["ddt"][1][at] = du.stored(store)
        by = (T, -1, per, N)
        for k, t in (("dB", g * (delta * xs)[..., None]), ("dC", h * ds[..., None])):
            t = Num(t.v.reshape(by), t.e.reshape(by), unit).sum(2)
            shared[k][0][at], shared[k][1][at] = t.stored(store)
        sums["dA"].append(q * delta[..., None])
        sums["dD"].append(ds * xs)
        sums["dbias"].append(du)
    outs["last"] = (last, laste)
    if dy is None:
        return outs
    outs.update(shared, dh0=(dh0, dh0e))
    for k, parts in sums.items():
        if not parts:
            shape = (d, N) if k == "dA" else (d,)
            outs[k] = (np.zeros(shape), np.zeros(shape))
            continue
        v = Num(np.concatenate([p.v for p in parts]), np.concatenate([p.e for p in parts]), unit)
        outs[k] = v.sum(0).stored(own)
    return outs


# ----- norms -----

def root(x):
    """1 / sqrt(x)."""
    v = 1.0 / np.sqrt(x.v)
    return Num(v, 4 * x.u * v + x.e * v / (2 * x.v), x.u)


def _normed(u, w, eps):
    n = u.v.shape[1]
    rstd = root((u * u).sum(1) * (1.0 / n) + eps)[:, None]
    return u * rstd, rstd


def _back(hat, rstd, g):
    n = g.v.shape[1]
    return rstd * (g - hat * ((g * hat).sum(1) * (1.0 / n))[:, None])


def norm_in(x, w, res, scale, eps, dy=None, dr=None, unit=U32, store="f32", stream="f32"):
    own = "f64" if unit == U64 else "f32"
    X, W = Num(x, 0, unit), Num(w, 0, unit)
    r = X * scale if scale is not None else X
    r = r + res if res is not None else r
    hat, rstd = _normed(r, W, eps)
    out = {"y": (hat * W).stored(store), "r": r.stored(stream)}
    if dy is None:
        return out
    D = Num(dy, 0, unit)
    d = _back(hat, rstd, D * W)
    d = d + dr if dr is not None else d
    out["dres"] = d.stored(stream)
    out["dx"] = (d * scale if scale is not None else d).stored(store)
    out["dw"] = (D * hat).sum(0).stored(own)
    out["dscale"] = (d * X).sum(0).stored(own)
    return out


def norm_out(x, w, gate, res, scale, order, eps, dy=None, unit=U32, store="f32", stream="f32"):
    own = "f64" if unit == U64 else "f32"
    X, W = Num(x, 0, unit), Num(w, 0, unit)
    S = silu(Num(gate, 0, unit)) if gate is not None else Num(np.ones_like(x), 0, unit)
    first = order == "gate_first"
    u = X * S if first else X
    hat, rstd = _normed(u, W, eps)
    n = hat * W if first else hat * W * S
    y = n * scale if scale is not None else n
    out = {"y": (y + res if res is not None else y).stored(stream)}
    if dy is None:
        return out
    g = Num(dy, 0, unit)
    dn = g * scale if scale is not None else g
    du = _back(hat, rstd, dn * W if first else dn * W * S)
    slope = silu_slope(Num(gate, 0, unit)) if gate is not None else Num(np.zeros_like(x), 0, unit)
    out["dx"] = (du * S if first else du).stored(store)
    out["dgate"] = (du * X * slope if first else dn * hat * W * slope).stored(store)
    out["dw"] = (dn * hat if first else dn * hat * S).sum(0).stored(own)
    out["dscale"] = (g * n).sum(0).stored(own)
    return out

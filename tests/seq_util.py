"""Plain references, in 64 bits, of the recurrences along a sequence and of the
AdamW step, with bounds on how far a computation in fewer bits may be off
(numpy, no library code)."""
from __future__ import annotations

import numpy as np

U32, U64 = 2.0 ** -24, 2.0 ** -53
# half the spacing of the storage types, relative; and their smallest step / 2
STORE = {"f64": (2.0 ** -53, 0.0), "f32": (2.0 ** -24, 2.0 ** -150),
         "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def coefficients(x, gate, mode):
    if mode == "linear":
        return gate, x, np.ones_like(x)
    return sigmoid(gate), sigmoid(-gate) * x, sigmoid(-gate)


def spans(lead, offsets):
    """Index of each sequence in arrays of leading shape `lead`."""
    if offsets is None:
        return [(s, slice(None)) for s in range(lead[0])]
    return [(slice(int(a), int(b)),) for a, b in zip(offsets[:-1], offsets[1:])]


def recurrence(x, gate, h0, offsets, mode, dh=None, dlast=None, unit=U32, store="f32"):
    """Values and error bounds of every output: {name: (value, bound)}.

    Bounds: a computation in the unit roundoff `unit` makes at most K
    roundings per step on the way of any term into any sum, whichever way the
    products and sums are associated: the coefficient and the weight of x (6
    each, and 2 |g| for the exponential's argument), a product and a sum on
    the path, and as many again for a product of coefficients taken apart
    and for joining parts.  E_t = |a_t| E_{t-1} + K unit H_t with the majorant
    H_t = |a_t| H_{t-1} + |b_t| bounds the sum of them.  The reference's own
    error (64 bits) is counted by doubling K for fp64."""
    K = 20 + 2 * (np.abs(gate[np.isfinite(gate)]).max(initial=0.0) if mode == "sigmoid" else 0)
    K *= 2 if unit == U64 else 1
    ku = K * unit
    a, b, keep = coefficients(x, gate, mode)
    n = (len(offsets) - 1) if offsets is not None else x.shape[0]
    d = x.shape[-1]
    st = np.zeros((n, d)) if h0 is None else h0.copy()
    h, eh, before, eb = (np.zeros_like(x) for _ in range(4))
    last, elast = st.copy(), np.zeros_like(st)
    where = spans(x.shape, offsets)
    for s, at in enumerate(where):
        A, Bv = a[at], b[at]
        v, H, E = st[s].copy(), np.abs(st[s]), np.zeros(d)
        hh, he, hb, hbe = (np.zeros_like(A) for _ in range(4))
        for t in range(A.shape[0]):
            hb[t], hbe[t] = v, E
            v = A[t] * v + Bv[t]
            H = np.abs(A[t]) * H + np.abs(Bv[t])
            E = np.abs(A[t]) * E + ku * H
            hh[t], he[t] = v, E
        h[at], eh[at], before[at], eb[at] = hh, he, hb, hbe
        last[s], elast[s] = v, E
    r, tiny = STORE[store]
    own = STORE["f64" if unit == U64 else "f32"]

    def stored(v, e, to=(r, tiny)):
        return v, e + to[0] * (np.abs(v) + e) + to[1]

    out = {"h": stored(h, eh), "last": stored(last, elast, own)}
    if dh is None:
        return out
    dx, edx, dg, edg = (np.zeros_like(x) for _ in range(4))
    dh0, edh0 = np.zeros_like(st), np.zeros_like(st)
    for s, at in enumerate(where):
        A, D = a[at], dh[at]
        Kp, X, HB, HE = keep[at], x[at], before[at], eb[at]
        mu = np.zeros(d) if dlast is None else dlast[s].copy()
        M, E = np.abs(mu), np.zeros(d)
        gx, gxe, gg, gge = (np.zeros_like(A) for _ in range(4))
        for t in range(A.shape[0] - 1, -1, -1):
            lam, L = D[t] + mu, np.abs(D[t]) + M
            el = E + ku * L
            w = A[t] * Kp[t] if mode == "sigmoid" else np.ones(d)
            diff, size = (HB[t] - X[t], np.abs(HB[t]) + np.abs(X[t])) if mode == "sigmoid" else \
                (HB[t], np.abs(HB[t]))
            gx[t], gxe[t] = lam * Kp[t], (el + ku * L) * Kp[t]
            gg[t] = lam * diff * w
            gge[t] = (el * size + (L + el) * HE[t] + ku * L * size) * w
            mu, M, E = A[t] * lam, np.abs(A[t]) * L, np.abs(A[t]) * (el + ku * L)
        dx[at], edx[at], dg[at], edg[at] = gx, gxe, gg, gge
        dh0[s], edh0[s] = mu, E
    out["dx"], out["dgate"] = stored(dx, edx), stored(dg, edg)
    out["dh0"] = stored(dh0, edh0, own)
    return out


# ----- AdamW -----

def mix(x):
    x = np.asarray(x, dtype=np.uint64) & np.uint64(0xFFFFFFFF)
    m = np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B1)) & m
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0xBB67AE85)) & m
    return x ^ (x >> np.uint64(16))


def noise(seed, step, n):
    """32 random bits of each of the first n < 2^32 elements."""
    key = mix((seed & 0xFFFFFFFF) ^ int(mix((seed >> 32) ^ int(mix(step & 0xFFFFFFFF)))))
    e = np.arange(n, dtype=np.uint64)
    return mix(e * np.uint64(0x9E3779B1) + key)


def levels(x, add, top, least):
    """float32 values (whole blocks of 256) rounded to the 8-bit form: `add`
    (uint64) is added to each magnitude's pattern, the low 20 bits dropped, and
    the block's largest takes the code `top` or the one below; codes under
    `least` become `least`."""
    bits = (x.view(np.uint32) & 0x7FFFFFFF).astype(np.int64).reshape(-1, 256)
    fin = bits < 0x7F800000
    k = np.minimum((np.where(fin, bits, 0).max(1, keepdims=True) + 0xFFFFF) >> 20, 2039)
    base = np.maximum(k - top, 0)
    code = np.clip(((bits + add.astype(np.int64).reshape(-1, 256)) >> 20) - base, least, top)
    code = np.where(bits == 0, 0, code)
    val = np.where(code == 0, 0, (code + base) << 20).astype(np.uint32).view(np.float32)
    val = np.where(fin, val, np.float32(np.inf) if least else np.float32(np.nan))
    return np.copysign(val.reshape(-1), x)


def pad_to_blocks(parts):
    out = []
    for p in parts:
        p = np.asarray(p).reshape(-1)
        out.append(np.concatenate([p, np.zeros(-len(p) % 256, p.dtype)]))
    return np.concatenate(out) if out else np.zeros(0, np.float32)


def moments32(m, v, g, b1, b2):
    """m' and v' in float32, every operation rounded by itself."""
    f = np.float32
    with np.errstate(over="ignore", invalid="ignore"):
        return m * f(b1) + g * f(1 - b1), v * f(b2) + (g * g) * f(1 - b2)


def adamw64(p, m, v, g, step, lr, b1, b2, eps, wd):
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    up = lr / (1 - b1 ** step) * m / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p * (1 - lr * wd) - up, m, v, up

"""Plain float64 references of the gated linear recurrence, the group norm and the products in 8-bit integers, with
first-order bounds of what fp32 arithmetic may add (as in _layer_ref: u = 2^-24 an operation, 2 u for exp2, log2, the
reciprocal and the square roots)."""
import numpy as np

from ._layer_ref import HALF, U, check, sigmoid, tol  # noqa: F401


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def gate(v, nb=0.0):
    """sigmoid(v + bias) and its relative error.  The exponent -log2(e) (v + bias) is off by 2 u of its parts, which the
    exponential multiplies by ln 2 (log2(e) ln 2 = 1): 2 u (|v| + |bias|); exp2 2 u, the sum u, the reciprocal 2 u."""
    s = sigmoid(v + nb)
    return s, (2 * (np.abs(v) + np.abs(nb)) * (1 - s) + 5) * U


class Gated:
    """Everything a step has, (B, D, L), with relative errors d*."""

    def __init__(self, x, r, i, lam, rb, ib, power):
        col = lambda p: 0.0 if p is None else p[:, None]  # noqa: E731
        self.x = x
        self.rho, drho = gate(r, col(rb))
        self.iota, self.diota = gate(i, col(ib))
        sp = softplus(lam)
        # softplus: exp2 of a rounded product, the sum's rounding put back, log2 and a product: 10 u and |lam| u of e^lam
        dsp = (10 + 2 * np.abs(lam)) * U
        self.share, self.dshare = sigmoid(lam) / sp, dsp + (2 * np.abs(lam) + 6) * U
        self.rate = power * sp[:, None]
        self.q = self.rate * self.rho
        self.drho = drho
        self.dq = drho + dsp[:, None] + 2 * U
        self.a = np.exp(-self.q)
        self.da = self.q * (self.dq + 2 * U) + 2 * U
        v = -np.expm1(-2 * self.q)
        # derivative of log(1 - e^-2q) by log q: at most 1; series, products and the difference: 8 u; where it is a
        # difference (q >= 1/2) a's error counts by 2 a^2 / (1 - a^2) <= 1.17
        self.dv = self.dq + 8 * U + 1.2 * np.where(self.q >= 0.5, self.da, 0)
        self.beta, self.dbeta = np.sqrt(v), self.dv / 2 + 4 * U
        self.u = self.iota * x
        self.b = self.beta * self.u
        self.db = self.dbeta + self.diota + 2 * U


# Below the smallest normal float, 2^-126, 1 - a^2 = 2 q (and q itself) may be taken as 0: its root beta, which is then
# below 2^-63, and q / beta = beta / 2 are off by no more than their own size.
SHUT = 2.0 ** -63


# From one step to a later one: a product and a sum a step (a tile's own two among them, 128 steps and more apart); and
# once the levels of the scan, two roundings each: 4 in 16 lanes, 3 in a wave, up to 16 waves less one a level
LEVELS = 40 * U


def scan(a, b, h0, da, db, du):
    """States h, and bounds: the recurrence of the errors, fed by those of a and b and the steps' roundings."""
    B, D, L = a.shape
    h, m, e = (np.zeros((B, D)) for _ in range(3))
    if h0 is not None:
        h, m = h0.copy(), np.abs(h0)
    H, M, E, P = (np.empty((B, D, L)) for _ in range(4))
    rel = da + 3 * U
    for t in range(L):
        P[..., t] = h
        e = a[..., t] * (e + m * rel[..., t]) + np.abs(b[..., t]) * db[..., t] + du[..., t]
        h = a[..., t] * h + b[..., t]
        m = a[..., t] * m + np.abs(b[..., t])
        H[..., t], M[..., t], E[..., t] = h, m, e
        e = e + U * m
    return H, E + LEVELS * M, P


def gated_fwd(x, r, i, lam, rb, ib, power, h0):
    g = Gated(x, r, i, lam, rb, ib, power)
    h, err, _ = scan(g.a, g.b, h0, g.da, g.db, SHUT * np.abs(g.u))
    last, dlast = (h[..., -1], err[..., -1]) if x.shape[2] else (h0, 0 * h0)
    return {"y": (h, err), "h_last": (last, dlast)}


def gated_bwd(x, r, i, lam, rb, ib, power, h0, gy, gl):
    g = Gated(x, r, i, lam, rb, ib, power)
    B, D, L = x.shape
    h, dh, prev = scan(g.a, g.b, h0, g.da, g.db, SHUT * np.abs(g.u))
    dprev = np.concatenate([np.zeros((B, D, 1)), dh[..., :-1]], -1)
    # mu is a scan from the last step to the first, of gy with the next step's a
    nxt = np.concatenate([g.a[..., 1:], np.ones((B, D, 1))], -1)
    dn = np.concatenate([g.da[..., 1:], np.zeros((B, D, 1))], -1)
    mu, dmu, _ = scan(nxt[..., ::-1], gy[..., ::-1], gl, dn[..., ::-1], np.zeros_like(gy), np.zeros_like(gy))
    mu, dmu = mu[..., ::-1], dmu[..., ::-1]
    one, two = g.q / g.beta * g.a ** 2 * g.u, g.q * g.a * prev
    E = mu * (one - two)
    # q / beta and a twice, u, products; q, a, h
    dE = (dmu * (np.abs(one) + np.abs(two)) + np.abs(mu) * (
        np.abs(one) * (g.dq + g.dbeta + 2 * g.da + g.diota + 8 * U) + np.abs(two) * (g.dq + g.da + 6 * U)
        + g.q * g.a * dprev + SHUT * np.abs(g.u)))
    gr = E * (1 - g.rho)
    dgr = dE * (1 - g.rho) + np.abs(E) * (g.rho * g.drho + 2 * U)
    gu = mu * g.beta
    dgu = dmu * g.beta + np.abs(gu) * (g.dbeta + 2 * U) + SHUT * np.abs(mu)
    gx, dgx = gu * g.iota, dgu * g.iota + np.abs(gu * g.iota) * (g.diota + 2 * U)
    k = g.u * (1 - g.iota)
    gi = gu * k
    dgi = dgu * np.abs(k) + np.abs(gu) * (np.abs(k) * (g.diota + 4 * U) + np.abs(g.u) * (g.iota * g.diota + U))
    # sums: eight steps, a tile of at least 128 after the other, lanes, the batch
    n = (8 + L / 128 + 12 + B / 16 + 16) * U
    out = {"gx": (gx, dgx), "gr": (gr, dgr), "gi": (gi, dgi), "gh0": (
        g.a[..., 0] * mu[..., 0], g.a[..., 0] * (dmu[..., 0] + np.abs(mu[..., 0]) * (g.da[..., 0] + 2 * U)))}
    for name, v, dv in (("glam", E, dE), ("gr_bias", gr, dgr), ("gi_bias", gi, dgi)):
        s, ds = v.sum((0, 2)), dv.sum((0, 2)) + n * np.abs(v).sum((0, 2))
        if name == "glam":
            ds = g.share * (ds + np.abs(s) * (g.dshare + 3 * U))
            s = g.share * s
        out[name] = (s, ds)
    return out


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------
def silu(v):
    """silu, its derivative and the bound of the derivative's slope (below 0.5 + ..: 0.6)."""
    s = sigmoid(v)
    return v * s, s * (1 + v * (1 - s))


def _act_err(v, dv):
    s, d = silu(v)
    rel = (2 * np.abs(v) + 8) * U
    return np.abs(d) * dv + 0.6 * dv * dv + rel * np.abs(s) + 2 * U * np.abs(s), 0.6 * dv + rel * (np.abs(d) + np.abs(v)) + 4 * U


def norm(x, groups, w, bias, eps, act, z, gy=None):
    T, C = x.shape
    n = C // groups
    # of a sum: elements of a lane (at most 16), lanes of a wave 6 levels, 16 waves, the product with 1 / n
    K = (16 + 6 + 16 + 3) * U
    X = x.reshape(T, groups, n)
    mean = X.mean(-1, keepdims=True)
    dmean = K * np.abs(X).mean(-1, keepdims=True)
    c = X - mean
    dc = dmean + U * np.abs(c)
    var = (c * c).mean(-1, keepdims=True)
    dvar = (2 * np.abs(c) * dc + dc * dc).mean(-1, keepdims=True) + K * var
    rstd = 1 / np.sqrt(var + eps)
    drstd = 0.5 * dvar / (var + eps) + 4 * U                         # relative
    xh = c * rstd
    dxh = rstd * dc + np.abs(xh) * (drstd + U)
    xh, dxh, W = xh.reshape(T, C), dxh.reshape(T, C), np.ones(C) if w is None else w
    v = xh * W + (0 if bias is None else bias)
    dv = np.abs(W) * dxh + U * np.abs(v)
    if act:
        u, du1 = silu(v)
        du, ddu1 = _act_err(v, dv)
    else:
        u, du1, du, ddu1 = v, np.ones_like(v), dv, 0 * dv
    if z is not None:
        sz, dsz1 = silu(z)
        esz, edsz1 = _act_err(z, 0 * z)
    else:
        sz, esz = np.ones_like(u), 0 * u
    out = {"y": (u * sz, du * np.abs(sz) + np.abs(u) * esz + 2 * U * np.abs(u * sz))}
    if gy is None:
        return out
    if z is not None:
        gz = gy * u * dsz1
        out["gz"] = (gz, np.abs(gy) * (du * np.abs(dsz1) + np.abs(u) * edsz1) + 4 * U * np.abs(gz))
    gu = gy * sz
    dgu = np.abs(gy) * esz + 2 * U * np.abs(gu)
    gv = gu * du1
    dgv = dgu * np.abs(du1) + np.abs(gu) * ddu1 + 2 * U * np.abs(gv)
    # sums over the rows: a wave's one after the other, the waves, the workgroups
    n2 = (T / 8 + 8 + 64 + 16) * U
    out["gbias"] = (gv.sum(0), dgv.sum(0) + n2 * np.abs(gv).sum(0))
    out["gw"] = ((gv * xh).sum(0), (dgv * np.abs(xh) + np.abs(gv) * dxh).sum(0) + n2 * np.abs(gv * xh).sum(0))
    gh, dgh = gv * W, dgv * np.abs(W) + U * np.abs(gv * W)
    r = lambda a: a.reshape(T, groups, n)  # noqa: E731
    gh, dgh, xh, dxh = r(gh), r(dgh), r(xh), r(dxh)
    m0, m1 = gh.mean(-1, keepdims=True), (gh * xh).mean(-1, keepdims=True)
    dm0 = dgh.mean(-1, keepdims=True) + K * np.abs(gh).mean(-1, keepdims=True)
    dm1 = (dgh * np.abs(xh) + np.abs(gh) * dxh).mean(-1, keepdims=True) + K * np.abs(gh * xh).mean(-1, keepdims=True)
    inner = gh - m0 - xh * m1
    dinner = dgh + dm0 + dxh * np.abs(m1) + np.abs(xh) * dm1 + 3 * U * (np.abs(gh) + np.abs(m0) + np.abs(xh * m1))
    out["gx"] = ((rstd * inner).reshape(T, C), (rstd * (dinner + np.abs(inner) * (drstd + U))).reshape(T, C))
    return out


# ---------------------------------------------------------------------------
# products in 8-bit integers
# ---------------------------------------------------------------------------
TINY8, TOP8 = 2.0 ** -100, float.fromhex("0x1.020406p+121")


def pack(x):
    """The 8-bit form of rows, bit for bit: float32 operations, each rounded once."""
    x = x.astype(np.float32)
    amax = np.abs(x).max(1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
    bad, zero = ~np.isfinite(amax), amax < np.float32(TINY8)
    safe = np.where(bad | zero, np.float32(1), amax).astype(np.float32)
    scale = np.minimum(safe / np.float32(127), np.float32(TOP8))
    inv = np.where(bad | zero, np.float32(0), np.float32(127) / safe)
    scale = np.where(bad, np.float32(np.nan), np.where(zero, np.float32(0), scale))
    with np.errstate(invalid="ignore"):
        q = np.rint(np.where(bad[:, None], np.float32(0), x) * inv[:, None].astype(np.float32))
    return q.astype(np.int8), scale.astype(np.float32)


def mm8(x8, xs, w8, ws, bias):
    """The sum is exact, its rounding to float32 u, the scales' product u, the last step u of the result."""
    acc = x8.astype(np.float64) @ w8.astype(np.float64).T   # whole numbers below 2^53: exact
    p = acc * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    y = p + (0 if bias is None else bias)
    return y, 2.1 * U * np.abs(p) + U * np.abs(y)

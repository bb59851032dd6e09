"""Plain float64 references of the short convolution, the 8-bit checkpoints and the packed-row forms, step by step,
with first-order bounds of what fp32 arithmetic may add.

Every reference takes float64 arrays that hold exactly the values of the streams under test and returns, next to each
result, `err`: a bound of the error of a computation in fp32 whose operations are rounded to u = 2^-24 (exp2 and the
reciprocal, whose hardware forms are accurate to one unit in the last place, to 2 u).  `tol` adds the output's own
rounding: half a step of its type, eps / 2 relative (bf16 2^-8, fp32 2^-24).
"""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
BLOCK = 64


def tol(ref, err, dtype):
    """Bound of |output - ref|: the fp32 error and its rounding to the output's type (of a value up to err away)."""
    return err + HALF[dtype] * (np.abs(ref) + err) + 1e-37


def check(name, got, ref, err, dtype):
    g = np.asarray(got.detach().cpu().double().numpy())
    assert g.shape == ref.shape, f"{name}: shape {g.shape} against {ref.shape}"
    assert np.array_equal(np.isnan(g), np.isnan(ref)), f"{name}: NaN in other places"
    fin = np.isfinite(ref)
    assert np.array_equal(g[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)]), f"{name}: infinities"
    over = np.abs(g[fin] - ref[fin]) - tol(ref, err, dtype)[fin]
    assert not (over > 0).any(), (f"{name}: {int((over > 0).sum())} of {over.size} elements beyond their bound, "
                                  f"worst by {over.max():.3e}")


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def silu_err(p, dp):
    """Error of p * sigmoid(p) from an error dp of p: its slope is below 1.1; the product with log2 e and its
    rounding put 2 |p| u into the exponent, exp2 2u, the sum u, the reciprocal 2u, the product u."""
    return 1.1 * dp + (2 * np.abs(p) + 6) * U * np.abs(p * sigmoid(p))


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------
def conv_pre(x, w, bias, init):
    B, D, L = x.shape
    W = w.shape[1]
    e = np.concatenate([np.zeros((B, D, W - 1)) if init is None else init, x], -1)
    p = np.zeros((B, D, L))
    m = np.zeros((B, D, L))
    if bias is not None:
        p += bias[:, None]
        m += np.abs(bias)[:, None]
    for t in range(L):
        p[..., t] += (w * e[..., t:t + W]).sum(-1)
        m[..., t] += np.abs(w * e[..., t:t + W]).sum(-1)
    return e, p, (W + 1) * U * m


def conv_fwd(x, w, bias, init, silu):
    """y and its bound, and the last W-1 inputs."""
    e, p, dp = conv_pre(x, w, bias, init)
    last = e[..., x.shape[2]:]
    return (p * sigmoid(p), silu_err(p, dp), last) if silu else (p, dp, last)


def conv_bwd(x, w, bias, init, silu, gy, glast):
    """dict of (gradient, bound)."""
    B, D, L = x.shape
    W = w.shape[1]
    e, p, dp = conv_pre(x, w, bias, init)
    if silu:
        s = sigmoid(p)
        gp = gy * s * (1 + p * (1 - s))
        # the slope's own slope is below 1/2; its terms are products of factors up to 1 + |p|
        dgp = np.abs(gy) * (0.5 * dp + (4 * np.abs(p) + 16) * U)
    else:
        gp, dgp = gy.copy(), np.zeros_like(gy)
    ge, dge = np.zeros_like(e), np.zeros_like(e)
    gw, dgw = np.zeros((D, W)), np.zeros((D, W))
    # a lane adds its runs of 8 in turn, 256 lanes a workgroup at least 1 run each, then lanes and parts
    depth = min(B * L, 8 * -(-(B * -(-L // 8)) // 256) + 1040) + 16
    for k in range(W):
        ge[..., k:k + L] += w[:, k, None] * gp
        dge[..., k:k + L] += np.abs(w[:, k, None]) * (dgp + (W + 2) * U * np.abs(gp))
        gw[:, k] = (gp * e[..., k:k + L]).sum((0, 2))
        dgw[:, k] = (np.abs(e[..., k:k + L]) * (dgp + depth * U * np.abs(gp))).sum((0, 2))
    if glast is not None:
        ge[..., L:] += glast
        dge[..., L:] += (W + 2) * U * np.abs(glast)
    return {"ginit": (ge[..., :W - 1], dge[..., :W - 1]), "gx": (ge[..., W - 1:], dge[..., W - 1:]),
            "gw": (gw, dgw), "gbias": (gp.sum((0, 2)), (dgp + depth * U * np.abs(gp)).sum((0, 2)))}


# ---------------------------------------------------------------------------
# 8-bit checkpoints (defined in fp32: exact)
# ---------------------------------------------------------------------------
def pack(x):
    """(whole numbers, scales) of x (B, D, L) float32."""
    B, D, L = x.shape
    nb = -(-L // BLOCK)
    q = np.zeros((B, D, L), np.int8)
    s = np.zeros((B, D, nb), np.float32)
    for i in range(nb):
        v = x[..., i * BLOCK:(i + 1) * BLOCK].astype(np.float32)
        amax = np.abs(v).max(-1, keepdims=True)
        bad = ~np.isfinite(amax)
        small = ~bad & (amax < np.float32(2.0 ** -100))
        ok = np.where(bad | small, np.float32(1), amax)
        n = np.where(bad | small, np.float32(0), np.rint(np.where(bad, np.float32(0), v) * (np.float32(127) / ok)))
        q[..., i * BLOCK:(i + 1) * BLOCK] = n.astype(np.int8)
        s[..., i] = np.where(bad, np.float32("nan"), np.where(small, np.float32(0), ok / np.float32(127)))[..., 0]
    return q, s


def unpack(q, s):
    """The values a checkpoint stands for, float32 (each product rounded once)."""
    return (q.astype(np.float32) * np.repeat(s, BLOCK, -1)[..., :q.shape[-1]]).astype(np.float32)


# ---------------------------------------------------------------------------
# packed rows
# ---------------------------------------------------------------------------
def owners(T, S, slots, seq_start, slot):
    """[(sequence, first row, end, slot)] of the sequences that own rows and a slot."""
    seen, got = set(), []
    for s in range(S):
        v = s if slot is None else int(slot[s])
        first, end = (s, s + 1) if seq_start is None else (int(seq_start[s]), int(seq_start[s + 1]))
        if 0 <= v < slots and v not in seen:
            if end > first:
                got.append((s, first, end, v))
        seen.add(v)
    return got


def tokens_conv(x, w, bias, silu, pool, seq_start, slot, fresh, y):
    """(y, bound, pool), y and pool copies updated by the call."""
    y, pool, err = y.copy(), pool.copy(), np.zeros_like(y)
    S = len(x) if seq_start is None else len(seq_start) - 1
    for s, a, b, v in owners(len(x), S, len(pool), seq_start, slot):
        init = np.zeros_like(pool[v]) if fresh is not None and fresh[s] else pool[v]
        o, d, last = conv_fwd(x[a:b].T[None], w, bias, init[None], silu)
        y[a:b], err[a:b], pool[v] = o[0].T, d[0].T, last[0]
    return y, err, pool


def tokens_scan(delta, x, A, Bm, C, skip, z, bias, softplus, pool, seq_start, slot, fresh, y):
    """(y, bound, pool, bound)."""
    y, pool, ye, pe = y.copy(), pool.copy(), np.zeros_like(y), np.zeros_like(pool)
    N = A.shape[1]
    S = len(x) if seq_start is None else len(seq_start) - 1
    for s, a, b, at in owners(len(x), S, len(pool), seq_start, slot):
        h = np.zeros_like(pool[at]) if fresh is not None and fresh[s] else pool[at].copy()
        hm, he = np.abs(h), np.zeros_like(h)
        for t in range(a, b):
            dl = delta[t] + (0 if bias is None else bias)
            de = 2 * U * (np.abs(delta[t]) + (0 if bias is None else np.abs(bias)))   # of the sum, absolute
            if softplus:   # its slope is below 1 and below itself; the exponent's 2 |v| u and ten roundings
                v = dl
                dl = np.logaddexp(v, 0)
                de = np.minimum(de, de * dl) + (2 * np.abs(v) + 10) * U * dl
            dl, de = dl[:, None], de[:, None]
            xt = x[t][:, None]
            f = np.exp(dl * A)
            term = dl * xt * Bm[t]
            # the exponent: A log2 e, the product and the step size's own error; exp2 2u; the fma u
            he = f * he + f * hm * (np.abs(A) * (4 * U * np.abs(dl) + de) + 3 * U) \
                + np.abs(xt * Bm[t]) * (de + 3 * U * np.abs(dl))
            h = f * h + term
            hm = f * hm + np.abs(term)
            # states that cross ranges of rows decay by exp(A sum delta) at once: u a step in the exponent,
            # at most (rows of a range) u / e of the state in all
            he = he + U * hm
            o = (C[t] * h).sum(1)
            oe = (np.abs(C[t]) * he).sum(1) + (N + 2) * U * (np.abs(C[t]) * hm).sum(1) \
                + 1024 * U * 0.37 * (np.abs(C[t]) * np.abs(h)).sum(1)
            if skip is not None:
                o = o + skip * x[t]
                oe = oe + 2 * U * np.abs(skip * x[t])
            if z is not None:
                g = z[t] * sigmoid(z[t])
                oe = np.abs(g) * oe + np.abs(o) * (silu_err(z[t], 0) + U * np.abs(g))
                o = o * g
            y[t], ye[t] = o, oe
        pool[at], pe[at] = h, he + 1024 * U * 0.37 * np.abs(h)
    return y, ye, pool, pe

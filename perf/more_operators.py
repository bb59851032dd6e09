"""Timed cases of the operators of a gated recurrent layer: the gated linear recurrence over training streams (forward
and backward) and over packed rows with a pool of states, the group norm of its rows with activation and gate (forward
and backward), and the serving layer's projections as products of 8-bit integers with scales for each token and channel.

A case's ``kind`` names its operator:

gated   training: the recurrence's states and every gradient, streams (B, D, L)
tgated  serving: the recurrence over the packed rows of a batch of sequences (or one row each)
norm    group norm of rows (T, C), channels last, with activation and gate; with ``train`` every gradient too
mm8     rows to 8-bit integers with a scale a row, and their product with 8-bit weights that have a scale a channel
"""
import math

import torch

own = False

DEV = torch.device("cuda" if torch.cuda.is_available() else "cpu")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
POWER = 8.0          # decay at a wide open gate: e^(-POWER softplus(lam))
EPS = 1e-5
TINY = 2.0 ** -100   # rows whose largest magnitude is below this are held as zeros


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a small layer with an odd number of channels and steps, carried on from a previous segment
        dict(name="gated_odd", kind="gated", B=2, D=195, L=517, dtype="f32", state=True),
        # a layer of the benchmark's size (B=8 D=2048 L=4096)
        dict(name="gated_layer", kind="gated", B=8, D=2048, L=4096, dtype="bf16", state=False),
        # one long sequence, as in the benchmark's impulse workload (B=1 D=1024 L=128000)
        dict(name="gated_long", kind="gated", B=1, D=1024, L=128000, dtype="f32", state=True),
        # prompts of very different lengths entering a server together
        dict(name="tgated_prompts", kind="tgated", T=8192, S=13, D=4096, dtype="bf16", step=False),
        # a few short prompts through a small layer, in fp32
        dict(name="tgated_odd", kind="tgated", T=333, S=5, D=200, dtype="f32", step=False),
        # one token for each sequence of a decoding batch with some of its places empty
        dict(name="tgated_step", kind="tgated", T=64, S=64, D=2048, dtype="bf16", step=True),
        # the norm and gate in front of a layer's output projection, in training
        dict(name="norm_layer", kind="norm", T=16384, C=2048, G=32, dtype="bf16", silu=False, gate=True, train=True),
        # an odd layer: groups that are no whole vectors, activation instead of a gate
        dict(name="norm_odd", kind="norm", T=777, C=195, G=3, dtype="f32", silu=True, gate=False, train=True),
        # a projection of a whole batch of prompts
        dict(name="mm8_prompts", kind="mm8", T=8192, K=4096, N=8192, dtype="bf16", bias=False),
        # a projection of a decoding batch
        dict(name="mm8_batch", kind="mm8", T=64, K=4096, N=2048, dtype="bf16", bias=True),
        # a projection of one token
        dict(name="mm8_one", kind="mm8", T=1, K=2048, N=4096, dtype="bf16", bias=False),
        # a small layer whose rows are no whole vectors, in fp32
        dict(name="mm8_odd", kind="mm8", T=333, K=515, N=1999, dtype="f32", bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(("gated", "tgated", "norm", "mm8"))
    dtype = rng.choice(("f32", "bf16"))
    if kind == "gated":
        L = _log(rng, 1, 16384)
        D = _log(rng, 16, 2048)
        return dict(kind=kind, B=rng.randint(1, max(1, min(8, 33554432 // (L * D)))), D=D, L=L, dtype=dtype,
                    state=rng.random() < 0.4)
    if kind == "tgated":
        D = _log(rng, 64, 4096)
        step = rng.random() < 0.4
        S = _log(rng, 1, 256)
        T = S
        if not step:
            T = _log(rng, 4, 8192)
            S = rng.randint(1, min(T, 24))
        return dict(kind=kind, T=T, S=S, D=D, dtype=dtype, step=step)
    if kind == "norm":
        T = _log(rng, 1, 16384)
        G = _log(rng, 1, 64)
        per = _log(rng, 4, 512)
        per = per // 8 * 8 if per >= 16 and rng.random() < 0.7 else per
        while T * G * per > 33554432:
            T = T // 2
        return dict(kind=kind, T=T, C=G * per, G=G, dtype=dtype, silu=rng.random() < 0.5, gate=rng.random() < 0.5,
                    train=rng.random() < 0.7)
    K = _log(rng, 64, 8192)
    N = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        K, N = -(-K // 64) * 64, -(-N // 64) * 64
    T = _log(rng, 1, 8192)
    while T * K * N > 8192 * 4096 * 8192:
        T = T // 2
    return dict(kind=kind, T=T, K=K, N=N, dtype=dtype, bias=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 23)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["kind"] == "norm":
        T, C = case["T"], case["C"]
        # groups with means of their own, rows of different sizes, as a scan leaves them
        s["x"] = ((randn(T, C) + 0.5 * randn(C)) * torch.exp(0.5 * randn(T, 1))).to(dt)
        s["z"] = randn(T, C).to(dt) if case["gate"] else None
        s["w"] = 1 + 0.1 * randn(C)
        s["bias"] = 0.1 * randn(C)
        s["gy"] = randn(T, C).to(dt) if case["train"] else None
        return s
    if case["kind"] == "mm8":
        T, K, N = case["T"], case["K"], case["N"]
        s["x"] = (randn(T, K) * torch.exp(0.5 * randn(K))).to(dt)   # columns of different sizes
        w = randn(N, K)
        s["w8_scale"] = w.abs().amax(1) / 127
        s["w8"] = torch.round(w / s["w8_scale"][:, None]).to(torch.int8)
        s["w8_scale"] = s["w8_scale"] / math.sqrt(K)
        s["bias"] = 0.1 * randn(N) if case["bias"] else None
        return s

    D = case["D"]
    s["lam"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * rand(D))))   # softplus(lam) of 0.001 to 0.105
    s["r_bias"], s["i_bias"] = 0.5 * randn(D), 0.5 * randn(D)
    if case["kind"] == "gated":
        B, L = case["B"], case["L"]
        s["x"] = (randn(B, D, L) * torch.exp(0.5 * randn(D, 1))).to(dt)
        s["r"], s["i"] = randn(B, D, L).to(dt), randn(B, D, L).to(dt)
        s["gy"] = randn(B, D, L).to(dt)
        s["h0"] = randn(B, D) if case["state"] else None
        s["gh_last"] = randn(B, D) if case["state"] else None
        return s

    T, S = case["T"], case["S"]
    if case["step"]:
        # a captured decoding batch has a fixed size: every eighth place is empty (slot -1) and leaves its row as it was
        s["seq_start"], s["fresh"] = None, None
        slots = S + S // 4 + 1
        slot = torch.randperm(slots, generator=g, device=DEV)[:S].to(torch.int32)
        places = torch.arange(S, device=DEV)
        slot[(places % 8 == 5) & (places > 0)] = -1
    else:
        # lengths of very different sizes, at least one token each
        cut = torch.sort(torch.randperm(T - 1, generator=g, device=DEV)[: S - 1] + 1).values if S > 1 else \
            torch.zeros(0, dtype=torch.int64, device=DEV)
        s["seq_start"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), cut,
                                    torch.full((1,), T, dtype=torch.int64, device=DEV)]).to(torch.int32)
        slots = S + 3
        slot = torch.randperm(slots, generator=g, device=DEV)[:S].to(torch.int32)
        s["fresh"] = rand(S) < 0.5    # the others carry on from a state in the pool
    s["slot"] = slot
    gates = randn(T, 2 * D).to(dt)    # one projection's output, read as two views
    s["r"], s["i"] = gates[:, :D], gates[:, D:]
    s["x"] = randn(T, D).to(dt)
    s["y"] = torch.zeros(T, D, dtype=dt, device=DEV)
    s["pool"] = randn(slots, D)
    return s


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    kind = case["kind"]
    if kind == "gated":   # x, r, i read and y written; gy read and three gradients written
        n, rows = case["B"] * case["D"] * case["L"], case["B"] * case["D"]
        return {"bytes": 8 * n * e + (16 * rows if case["state"] else 4 * rows) + 24 * case["D"], "flops": 80 * n}
    if kind == "tgated":
        T, S, D = case["T"], case["S"], case["D"]
        if case["step"]:
            T = S = S - (S + 2) // 8   # without the empty places
        return {"bytes": 4 * T * D * e + 8 * S * D + 12 * D + 4 * S, "flops": 30 * T * D}
    if kind == "norm":    # x (and z) read, y written; gy read, gx (and gz) written
        n = case["T"] * case["C"]
        streams = 2 + case["gate"] + ((2 + case["gate"]) if case["train"] else 0)
        return {"bytes": streams * n * e + (16 if case["train"] else 8) * case["C"], "flops": (40 if case["train"] else 15) * n}
    T, K, N = case["T"], case["K"], case["N"]
    return {"bytes": T * K * (e + 1) + N * K + T * N * e + 4 * T + (8 if case["bias"] else 4) * N,
            "flops": 2 * T * K * N + 5 * T * K}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _gates(s, ch):
    """The opened gates and what they make of the decay: rho, iota, q = -log a, a, beta.  ``ch``: a parameter (D,) laid
    beside the streams' channels."""
    rho = _sigmoid(s["r"].float() + ch(s["r_bias"]))
    iota = _sigmoid(s["i"].float() + ch(s["i_bias"]))
    q = ch(POWER * torch.log1p(torch.exp(s["lam"]))) * rho
    return rho, iota, q, torch.exp(-q), torch.sqrt(-torch.expm1(-2 * q))


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the last dimension, h before it zero; a and b are used up."""
    k = 1
    while k < b.shape[-1]:   # the maps h -> a h + b of 2k steps from those of k
        b[..., k:] = b[..., k:] + a[..., k:] * b[..., :-k]
        a[..., k:] = a[..., k:] * a[..., :-k]
        k *= 2
    return b


def _gated(s):
    dt, x = s["x"].dtype, s["x"].float()
    rho, iota, q, a, beta = _gates(s, lambda p: p[:, None])
    u = iota * x
    b = beta * u
    if s["h0"] is not None:
        b[..., 0] += a[..., 0] * s["h0"]
    h = _scan(a.clone(), b)
    before = torch.zeros_like(h)   # the state that each step begins with
    before[..., 1:] = h[..., :-1]
    if s["h0"] is not None:
        before[..., 0] = s["h0"]
    mu = s["gy"].float().clone()
    if s["gh_last"] is not None:
        mu[..., -1] += s["gh_last"]
    after = torch.zeros_like(a)
    after[..., :-1] = a[..., 1:]
    mu = _scan(after.flip(-1), mu.flip(-1)).flip(-1)
    e = mu * (torch.where(beta > 0, q / beta, 0) * a * a * u - q * a * before)
    gr = e * (1 - rho)
    gu = mu * beta
    gi = gu * x * iota * (1 - iota)
    share = _sigmoid(s["lam"]) / torch.log1p(torch.exp(s["lam"]))
    return {"y": h.to(dt), "h_last": h[..., -1].clone(), "gx": (gu * iota).to(dt), "gr": gr.to(dt), "gi": gi.to(dt),
            "glam": share * e.sum((0, 2)), "gr_bias": gr.sum((0, 2)), "gi_bias": gi.sum((0, 2)), "gh0": a[..., 0] * mu[..., 0]}


def _tgated(s):
    T, slot = s["T"], s["slot"]
    rho, iota, q, a, beta = _gates(s, lambda p: p)
    h = beta * iota * s["x"].float()
    h0 = s["pool"][slot.long().clamp(min=0)]
    if s["step"]:
        h += a * h0
        last = h
    else:
        start = s["seq_start"][:-1].long()
        h[start] += a[start] * torch.where(s["fresh"][:, None], torch.zeros_like(h0), h0)
        a[start] = 0
        h = _scan(a.T.contiguous(), h.T.contiguous()).T
        last = h[s["seq_start"][1:].long() - 1]
    held = slot >= 0
    s["pool"][slot[held].long()] = last[held]
    if s["step"]:
        s["y"].copy_(torch.where(held[:, None], h.to(s["y"].dtype), s["y"]))
    else:
        s["y"].copy_(h)
    return {"y": s["y"], "pool": s["pool"]}


def _norm(s):
    T, C, G, dt = s["T"], s["C"], s["G"], s["x"].dtype
    x = s["x"].float().view(T, G, C // G)
    x = x - x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = (x * rstd).view(T, C)
    v = xh * s["w"] + s["bias"]
    sv = _sigmoid(v) if s["silu"] else None
    u = v * sv if s["silu"] else v
    out = {}
    if s["gate"]:
        z = s["z"].float()
        sz = _sigmoid(z)
    out["y"] = (u * z * sz if s["gate"] else u).to(dt)
    if not s["train"]:
        return out
    gy = s["gy"].float()
    if s["gate"]:
        out["gz"] = (gy * u * sz * (1 + z * (1 - sz))).to(dt)
        gy = gy * z * sz
    gv = gy * sv * (1 + v * (1 - sv)) if s["silu"] else gy
    gh = (gv * s["w"]).view(T, G, C // G)
    xg = xh.view(T, G, C // G)
    gx = rstd * (gh - gh.mean(-1, keepdim=True) - xg * (gh * xg).mean(-1, keepdim=True))
    return {**out, "gx": gx.reshape(T, C).to(dt), "gw": (gv * xh).sum(0), "gbias": gv.sum(0)}


def _mm8(s):
    x = s["x"].float()
    amax = x.abs().amax(1, keepdim=True)
    held = amax >= TINY
    steps = torch.full_like(amax, 127)   # as a tensor: both quotients are then rounded once
    scale = torch.where(held, amax / steps, 0)
    x8 = torch.round(x * torch.where(held, steps / amax, 0))
    y = (x8 @ s["w8"].float().T) * scale * s["w8_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"x8": x8.to(torch.int8), "x8_scale": scale.squeeze(1), "y": y.to(s["x"].dtype)}


def run(s):
    if own:
        return _own(s)
    return {"gated": _gated, "tgated": _tgated, "norm": _norm, "mm8": _mm8}[s["kind"]](s)


# ---------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------
def _own(s):
    import selective_state_space_chunked_amd as ssm
    kind = s["kind"]
    if kind == "norm":
        par = dict(x=s["x"], groups=s["G"], w=s["w"], bias=s["bias"], eps=EPS, silu=s["silu"], z=s["z"])
        f = ssm.group_norm_fwd(**par)
        return {**f, **ssm.group_norm_bwd(gy=s["gy"], **par)} if s["train"] else f
    if kind == "mm8":
        f = ssm.tokens_pack8(s["x"])
        y = ssm.tokens_mm8(x8=f["x8"], x8_scale=f["x8_scale"], w8=s["w8"], w8_scale=s["w8_scale"], bias=s["bias"],
                           dtype=s["x"].dtype)
        return {**f, **y}
    par = dict(x=s["x"], r=s["r"], i=s["i"], lam=s["lam"], r_bias=s["r_bias"], i_bias=s["i_bias"], power=POWER)
    if kind == "gated":
        f = ssm.gated_fwd(h0=s["h0"], want_h_last=True, want_ckpt=True, **par)
        g = ssm.gated_bwd(gy=s["gy"], gh_last=s["gh_last"], h0=s["h0"], ckpt=f["ckpt"], **par)
        return {"y": f["y"], "h_last": f["h_last"], **g}
    f = ssm.tokens_gated(pool=s["pool"], seq_start=s["seq_start"], slot=s["slot"], fresh=s["fresh"], out={"y": s["y"]},
                         **par)
    return {"y": f["y"], "pool": s["pool"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _softplus64(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def _exact_gated(s):
    def steps_first(t):   # (B, D, L) to (L, B, D): a loop's step is one block
        return t.double().permute(2, 0, 1).contiguous()

    x, lam = steps_first(s["x"]), s["lam"].double()
    rho = torch.special.expit(steps_first(s["r"]) + s["r_bias"].double())
    iota = torch.special.expit(steps_first(s["i"]) + s["i_bias"].double())
    rate = POWER * _softplus64(lam)
    a = torch.exp(-rate * rho)
    beta = torch.sqrt(-torch.expm1(-2 * rate * rho))
    inp = beta * iota * x
    L, B, D = x.shape
    h = torch.empty(L + 1, B, D, dtype=torch.float64, device=x.device)
    h[0] = 0 if s["h0"] is None else s["h0"].double()
    for t in range(L):
        torch.addcmul(inp[t], a[t], h[t], out=h[t + 1])
    y, h_last = h[1:].permute(1, 2, 0).contiguous(), h[L].clone()
    mu = steps_first(s["gy"])
    if s["gh_last"] is not None:
        mu[L - 1] += s["gh_last"].double()
    for t in range(L - 1, 0, -1):
        mu[t - 1].addcmul_(a[t], mu[t])
    gh0 = a[0] * mu[0]
    gb = mu * beta
    # the decay's rate at a step is rate * rho: its derivative through a = e^-q and beta = sqrt(1 - e^-2q)
    gq = mu * (a * a / beta * iota * x - a * h[:L])
    glam = (gq * rho).sum((0, 1)) * POWER * torch.special.expit(lam)
    gr = gq * rate * rho * (1 - rho)
    gi = gb * x * iota * (1 - iota)
    back = [t.permute(1, 2, 0) for t in (gb * iota, gr, gi)]
    return {"y": y, "h_last": h_last, "gx": back[0], "gr": back[1], "gi": back[2], "glam": glam,
            "gr_bias": gr.sum((0, 1)), "gi_bias": gi.sum((0, 1)), "gh0": gh0}


def _exact_tgated(s):
    S = s["S"]
    start = s["seq_start"].tolist() if s["seq_start"] is not None else list(range(S + 1))
    slot, fresh = s["slot"].tolist(), s["fresh"].tolist() if s["fresh"] is not None else [False] * S
    y, pool = s["y"].double(), s["pool"].double()
    rate = POWER * _softplus64(s["lam"].double())
    q = rate * torch.special.expit(s["r"].double() + s["r_bias"].double())
    a = torch.exp(-q)
    b = torch.sqrt(-torch.expm1(-2 * q)) * torch.special.expit(s["i"].double() + s["i_bias"].double()) * s["x"].double()
    for n in range(S):
        if slot[n] < 0:
            continue
        h = torch.zeros_like(rate) if fresh[n] else pool[slot[n]].clone()
        for t in range(start[n], start[n + 1]):
            h = torch.addcmul(b[t], a[t], h)
            y[t] = h
        pool[slot[n]] = h
    return {"y": y, "pool": pool}


def _exact_norm(s):
    T, C, G = s["T"], s["C"], s["G"]
    leaves = {"gx": s["x"].double().requires_grad_(), "gw": s["w"].double().requires_grad_(),
              "gbias": s["bias"].double().requires_grad_()}
    if s["gate"]:
        leaves["gz"] = s["z"].double().requires_grad_()
    part = leaves["gx"].unflatten(1, (G, C // G))
    var, mean = torch.var_mean(part, dim=2, keepdim=True, correction=0)
    v = ((part - mean) * torch.rsqrt(var + EPS)).flatten(1) * leaves["gw"] + leaves["gbias"]
    if s["silu"]:
        v = v * torch.special.expit(v)
    if s["gate"]:
        v = v * leaves["gz"] * torch.special.expit(leaves["gz"])
    out = {"y": v.detach()}
    if s["train"]:
        out.update(zip(leaves, torch.autograd.grad(v, list(leaves.values()), s["gy"].double())))
    return out


def _exact_mm8(s):
    # the 8-bit form is defined in fp32: step and product are rounded to fp32, from exact products and quotients
    x = s["x"].double()
    big = x.abs().amax(1, keepdim=True)
    none = big < TINY
    big = big.masked_fill(none, 1.0)
    whole = (x * (127 / big).float().double()).float().round().double().masked_fill(none, 0.0)
    scale = (big / 127).float().double().masked_fill(none, 0.0)
    y = torch.mm(whole, s["w8"].double().T.contiguous()) * (scale * s["w8_scale"].double())
    if s["bias"] is not None:
        y += s["bias"].double()
    return {"x8": None, "x8_scale": scale[:, 0], "y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "tgated": _exact_tgated, "norm": _exact_norm, "mm8": _exact_mm8}[case["kind"]](s)

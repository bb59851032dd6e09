"""The short convolution, 8-bit activation checkpoints and the packed-row forms on the GPU, against float64 references
with bounds derived from the arithmetic (tests/_layer_ref.py)."""
import numpy as np
import pytest
import torch

import selective_state_space_chunked_amd as ssm

from . import _layer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    return np.random.default_rng(seed)


def dev(a, dtype="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DT[dtype]).to(DEV)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------
def conv_inputs(B, D, L, W, dtype, init, seed, view=False):
    r = gen(seed)
    t = dict(w=dev(r.normal(size=(D, W)) / W), bias=dev(r.normal(size=D) * 0.3))
    x = dev(r.normal(size=(B, D, L + 5)), dtype)
    gy = dev(r.normal(size=(B, D, L + 5)), dtype)
    if view:    # rows that start inside a wider buffer
        t["x"], gy = x[..., 3:3 + L], gy[..., 1:1 + L]
    else:
        t["x"], gy = x[..., :L].contiguous(), gy[..., :L].contiguous()
    t["init"] = dev(r.normal(size=(B, D, W - 1)), dtype) if init else None
    return t, gy, dev(r.normal(size=(B, D, W - 1)), dtype) if init else None


def conv_check(t, gy, glast, silu, dtype, x64=None, fwd=True, **src):
    B, D, L = gy.shape
    a = [f64(t["x"]) if x64 is None else x64, f64(t["w"]), f64(t["bias"]), f64(t["init"])]
    par = dict(w=t["w"], bias=t["bias"], init=t["init"], silu=silu)
    src = src or dict(x=t["x"])
    if fwd:
        f = ssm.conv_fwd(want_last=True, **src, **par, **({"dtype": DT[dtype]} if "ckpt8" in src else {}))
        y, err, last = R.conv_fwd(*a, silu)
        R.check("y", f["y"], y, err, dtype)
        R.check("last", f["last"], last, 0 * last, dtype)
    g = ssm.conv_bwd(gy=gy, glast=glast, **src, **par)
    for k, (ref, err) in R.conv_bwd(*a, silu, f64(gy), f64(glast)).items():
        R.check(k, g[k], ref, err, "f32" if k in ("gw", "gbias") else dtype)
    return g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("B,D,L,W", [(1, 1, 1, 4), (2, 3, 2, 4), (2, 5, 3, 2), (3, 7, 8, 3), (1, 40, 63, 4), (2, 9, 64, 2),
                                     (2, 6, 65, 3), (1, 33, 517, 4), (2, 3, 2048, 4), (1, 2, 2057, 3), (1, 5, 5003, 4)])
def test_conv(B, D, L, W, silu, dtype):
    t, gy, glast = conv_inputs(B, D, L, W, dtype, L % 2 == 1, B + D + L)
    conv_check(t, gy, glast, silu, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_views_and_outputs(dtype):
    """Inputs and outputs that are slices of wider buffers (nothing outside them is written), inputs shared by the
    batch, and each output alone."""
    t, gy, glast = conv_inputs(2, 5, 77, 4, dtype, True, 3, view=True)
    conv_check(t, gy, glast, True, dtype)
    par = dict(w=t["w"], bias=t["bias"], init=t["init"], silu=True)
    wide = torch.full((2, 5, 90), 7.0, dtype=DT[dtype], device=DEV)
    f = ssm.conv_fwd(x=t["x"], **par)
    ssm.conv_fwd(x=t["x"], out={"y": wide[..., 6:83]}, **par)
    assert torch.equal(wide[..., 6:83], f["y"])
    assert (wide[..., :6] == 7).all() and (wide[..., 83:] == 7).all()
    g = ssm.conv_bwd(gy=gy, glast=glast, x=t["x"], **par)
    for k in g:
        one = ssm.conv_bwd(gy=gy, glast=glast, x=t["x"], want=(k,), **par)
        assert set(one) == {k} and torch.equal(one[k], g[k]), k
    wide.fill_(7.0)
    ssm.conv_bwd(gy=gy, glast=glast, x=t["x"], want=(), out={"gx": wide[..., 6:83]}, **par)
    assert torch.equal(wide[..., 6:83], g["gx"]) and (wide[..., 83:] == 7).all() and (wide[..., :6] == 7).all()
    shared = dict(t, x=t["x"][:1].expand(2, 5, 77))
    conv_check(shared, gy, glast, True, dtype)
    last = ssm.conv_fwd(x=t["x"], want_y=False, want_last=True, **par)
    assert set(last) == {"last"} and torch.equal(last["last"], t["x"][..., -3:])


def test_conv_parts_and_determinism():
    """Few channels and long rows: the sums of gw and gbias come in parts, in one order every time."""
    t, gy, glast = conv_inputs(3, 2, 9001, 4, "f32", True, 9)
    g = conv_check(t, gy, glast, True, "f32", fwd=False)
    for _ in range(3):
        h = ssm.conv_bwd(gy=gy, glast=glast, x=t["x"], w=t["w"], bias=t["bias"], init=t["init"], silu=True)
        assert all(torch.equal(g[k], h[k]) for k in g)


@pytest.mark.parametrize("dtype,x8", [("f32", False), ("bf16", False), ("f32", True)])
@pytest.mark.parametrize("B,D,L,W", [(2, 3, 1999, 2), (3, 4, 4095, 3), (2, 3, 10241, 4), (1, 2, 10243, 4), (4, 2, 8193, 2),
                                     (7, 2, 510, 4), (3, 5, 2561, 4), (2, 3, 2562, 3),
                                     (3, 2, 513, 4), (2, 2, 514, 3), (2, 3, 2600, 4), (1, 4, 1000, 3)])
def test_conv_backward_of_long_rows(B, D, L, W, dtype, x8):
    """Rows of tiles of 512 steps: the last one whole, short by a little, or with one step or two."""
    t, gy, glast = conv_inputs(B, D, L, W, dtype, True, L)
    src, kept = {}, None
    if x8:
        k = ssm.ckpt8_pack(t["x"])
        src = dict(ckpt8=(k["x8"], k["x8_scale"]))
        kept = R.unpack(k["x8"].cpu().numpy(), k["x8_scale"].cpu().numpy()).astype(np.float64)
    conv_check(t, gy, glast, L % 4 != 1, dtype, x64=kept, fwd=False, **src)


def test_conv_parts_of_several_groups():
    """Channels and steps enough that a workgroup takes two groups of several parts, across rows."""
    t, gy, glast = conv_inputs(4, 1100, 4091, 4, "bf16", True, 11)
    conv_check(t, gy, glast, True, "bf16", fwd=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_conv_segments(dtype):
    """A sequence in two segments is the whole one: last becomes init, ginit becomes glast, bit for bit in the streams."""
    t, gy, _ = conv_inputs(2, 6, 203, 4, dtype, False, 21)
    par = dict(w=t["w"], bias=t["bias"], silu=True)
    whole = ssm.conv_fwd(x=t["x"], want_last=True, **par)
    wg = ssm.conv_bwd(gy=gy, x=t["x"], **par)
    a, b = t["x"][..., :88], t["x"][..., 88:]
    f1 = ssm.conv_fwd(x=a, want_last=True, **par)
    f2 = ssm.conv_fwd(x=b, init=f1["last"], want_last=True, **par)
    assert torch.equal(torch.cat([f1["y"], f2["y"]], -1), whole["y"]) and torch.equal(f2["last"], whole["last"])
    g2 = ssm.conv_bwd(gy=gy[..., 88:], x=b, init=f1["last"], **par)
    g1 = ssm.conv_bwd(gy=gy[..., :88], glast=g2["ginit"], x=a, **par)
    # where the segments meet, the carried gradient is rounded to the stream's type and added at another place
    mag = wg["gx"].float().abs() + g1["gx"].float().abs().max()
    lim = (4 * R.HALF[dtype] * mag + 1e-30)
    assert ((torch.cat([g1["gx"], g2["gx"]], -1).float() - wg["gx"].float()).abs() <= lim).all()


@pytest.mark.parametrize("silu", [False, True])
def test_conv_gradient_by_differences(silu):
    """The kernel's gradients against central differences of the kernel's own fp32 outputs."""
    t, gy, glast = conv_inputs(1, 2, 9, 4, "f32", True, 33)
    names = {"x": "gx", "w": "gw", "bias": "gbias", "init": "ginit"}

    def loss(over):
        a = {**t, **over}
        f = ssm.conv_fwd(x=a["x"], w=a["w"], bias=a["bias"], init=a["init"], silu=silu, want_last=True)
        return float((f["y"].double() * gy.double()).sum() + (f["last"].double() * glast.double()).sum())

    g = ssm.conv_bwd(gy=gy, glast=glast, x=t["x"], w=t["w"], bias=t["bias"], init=t["init"], silu=silu)
    h = 2.0 ** -7
    # outputs of order 1 carry about 10 u of fp32 error each, divided by 2 h; h^2 / 6 of a third derivative of a few
    lim = 40 * 10 * R.U * 8 / (2 * h) + 20 * h * h / 6
    for k, name in names.items():
        for i in np.ndindex(*t[k].shape):
            up, dn = t[k].clone(), t[k].clone()
            up[i] += h
            dn[i] -= h
            step = float(up[i].double() - dn[i].double())
            assert abs((loss({k: up}) - loss({k: dn})) / step - float(g[name][i])) < lim, (name, i)


def test_conv_non_finite_values_stay_in_their_window():
    """A NaN or infinity reaches the outputs whose window holds it, and no other row or step."""
    t, gy, _ = conv_inputs(2, 3, 40, 4, "f32", False, 4)
    clean = ssm.conv_fwd(x=t["x"], w=t["w"], bias=t["bias"], silu=False)["y"]
    x = t["x"].clone()
    x[0, 1, 17] = float("nan")
    x[1, 2, 39] = float("inf")
    y = ssm.conv_fwd(x=x, w=t["w"], bias=t["bias"], silu=False)["y"]
    assert torch.isnan(y[0, 1, 17:21]).all() and torch.isinf(y[1, 2, 39])
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[0, 1, 17:21] = False
    keep[1, 2, 39] = False
    assert torch.equal(y[keep], clean[keep])
    gyn = gy.clone()
    gyn[0, 0, 39] = float("nan")    # the last step: reaches gx of its window, not steps past the end
    g = ssm.conv_bwd(gy=gyn, x=t["x"], w=t["w"], bias=t["bias"], want=("gx",))["gx"]
    assert torch.isnan(g[0, 0, 36:]).all() and torch.isfinite(g[0, 0, :36]).all() and torch.isfinite(g[1]).all()


@pytest.mark.parametrize("over", [dict(B=0), dict(D=0), dict(L=0)])
def test_conv_empty(over):
    B, D, L = over.get("B", 2), over.get("D", 3), over.get("L", 5)
    w, bias = torch.ones(D, 4, device=DEV), torch.ones(D, device=DEV)
    x, st = torch.ones(B, D, L, device=DEV), torch.full((B, D, 3), 2.0, device=DEV)
    f = ssm.conv_fwd(x=x, w=w, bias=bias, init=st, want_last=True, want_ckpt8=True)
    g = ssm.conv_bwd(gy=x, glast=3 * st, x=x, w=w, bias=bias, init=st)
    assert f["y"].shape == (B, D, L) and torch.equal(f["last"], st) and torch.equal(g["ginit"], 3 * st)
    assert (g["gw"] == 0).all() and (g["gbias"] == 0).all()
    f = ssm.conv_fwd(x=x, w=w, want_last=True)
    assert (f["last"] == 0).all()


# ---------------------------------------------------------------------------
# 8-bit checkpoints
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,L", [(1, 1, 1), (2, 3, 63), (1, 5, 64), (2, 2, 65), (1, 3, 200), (2, 1, 4099)])
def test_ckpt8(B, D, L, dtype):
    """Equal to the definition, element for element: it is stated in fp32."""
    r = gen(L)
    x = dev(r.normal(size=(B, D, L)) * np.exp(r.normal(size=(B, D, 1)) * 3), dtype)
    got = ssm.ckpt8_pack(x)
    q, s = R.pack(x.float().cpu().numpy())
    assert np.array_equal(got["x8"].cpu().numpy(), q) and np.array_equal(got["x8_scale"].cpu().numpy(), s)
    v = R.unpack(q, s)
    assert np.array_equal(ssm.ckpt8_unpack(got["x8"], got["x8_scale"]).cpu().numpy(), v)
    as_bf16 = ssm.ckpt8_unpack(got["x8"], got["x8_scale"], dtype=torch.bfloat16)
    assert torch.equal(as_bf16.cpu(), torch.from_numpy(v).bfloat16())
    xf = x.double().cpu().numpy()
    assert (np.abs(v - xf) <= (0.5 + 2.0 ** -16) * np.repeat(s, 64, -1)[..., :L].astype(np.float64)).all()


def test_ckpt8_special_blocks():
    x = torch.ones(1, 1, 6 * 64, device=DEV)
    x[..., 64:128] = 0.0
    x[..., 128:192] *= 2.0 ** -101          # below the smallest block kept
    x[..., 192 + 5] = float("nan")
    x[..., 256 + 9] = float("-inf")
    x[..., 320:] *= 3.0e38
    p = ssm.ckpt8_pack(x)
    v = ssm.ckpt8_unpack(p["x8"], p["x8_scale"])[0, 0].view(6, 64)
    assert (v[0] == 1).all() and (v[1] == 0).all() and (v[2] == 0).all()
    assert torch.isnan(v[3]).all() and torch.isnan(v[4]).all() and torch.isfinite(v[5]).all()
    q, s = R.pack(x.cpu().numpy())
    assert np.array_equal(p["x8"].cpu().numpy(), q)
    assert np.array_equal(p["x8_scale"].cpu().numpy(), s, equal_nan=True)


def test_ckpt8_views():
    x = torch.randn(2, 7, 150, device=DEV)[:, 1:6, 3:140]
    p, q = ssm.ckpt8_pack(x), ssm.ckpt8_pack(x.contiguous())
    assert torch.equal(p["x8"], q["x8"]) and torch.equal(p["x8_scale"], q["x8_scale"])
    wide = torch.full((2, 5, 141), 7.0, device=DEV)
    ssm.ckpt8_unpack(p["x8"], p["x8_scale"], out=wide[..., 2:139])
    assert torch.equal(wide[..., 2:139], ssm.ckpt8_unpack(p["x8"], p["x8_scale"]))
    assert (wide[..., :2] == 7).all() and (wide[..., 139:] == 7).all()
    x8 = torch.zeros(3 + 2 * 5 * 137, dtype=torch.int8, device=DEV)[3:].view(2, 5, 137)   # odd address
    ssm.ckpt8_pack(x, out={"x8": x8})
    assert torch.equal(x8, q["x8"])
    x64 = torch.randn(1, 2, 128, device=DEV)
    x8 = torch.zeros(3 + 256, dtype=torch.int8, device=DEV)[3:].view(1, 2, 128)
    ssm.ckpt8_pack(x64, out={"x8": x8})
    ref = ssm.ckpt8_pack(x64)
    assert torch.equal(x8, ref["x8"])
    assert torch.equal(ssm.ckpt8_unpack(x8, ref["x8_scale"]), ssm.ckpt8_unpack(ref["x8"], ref["x8_scale"]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,L,W", [(1, 2, 1, 4), (2, 5, 71, 3), (1, 9, 512, 4), (2, 3, 2111, 2)])
def test_conv_from_its_checkpoint(B, D, L, W, dtype):
    """The checkpoint written by the forward pass is ckpt8_pack's; forward and backward from it are those of the values it
    stands for."""
    t, gy, glast = conv_inputs(B, D, L, W, dtype, True, L + W)
    par = dict(w=t["w"], bias=t["bias"], init=t["init"], silu=True)
    f = ssm.conv_fwd(x=t["x"], want_ckpt8=True, want_last=True, **par)
    p = ssm.ckpt8_pack(t["x"])
    plain = ssm.conv_fwd(x=t["x"], want_last=True, **par)
    assert torch.equal(f["x8"], p["x8"]) and torch.equal(f["x8_scale"], p["x8_scale"])
    assert torch.equal(f["y"], plain["y"]) and torch.equal(f["last"], plain["last"])
    kept = R.unpack(f["x8"].cpu().numpy(), f["x8_scale"].cpu().numpy()).astype(np.float64)
    conv_check(t, gy, glast, True, dtype, x64=kept, ckpt8=(f["x8"], f["x8_scale"]))


# ---------------------------------------------------------------------------
# packed rows
# ---------------------------------------------------------------------------
LENGTHS = {
    "one": [1], "long": [1500], "ragged": [1, 2, 3, 50, 0, 4, 129, 1, 1, 0, 300], "short": [1] * 70 + [2] * 5,
    "ends": [15, 1, 16, 17, 31, 33, 64, 2, 1, 65], "zero": [0, 0, 5, 0],
}


def sequences(lengths, seed, slots_more=3, empty=True, before=0):
    """seq_start, slot, fresh as numpy; with `empty` every fifth sequence (from the third) an empty place."""
    r = gen(seed)
    S = len(lengths)
    start = before + np.concatenate([[0], np.cumsum(lengths)])
    slot = r.permutation(S + slots_more)[:S].astype(np.int32)
    if empty:
        slot[2::5] = -1
    return start.astype(np.int32), slot, r.random(S) < 0.5, S + slots_more


def tok_rows(T, D, dtype, r, view, poison):
    """Rows (T, D), a slice of wider ones with `view`; rows in `poison` are NaN."""
    wide = r.normal(size=(T, D + 11 if view else D))
    wide[poison] = np.nan
    t = dev(wide, dtype)
    return t[:, 3:3 + D] if view else t


def unowned(T, owned):
    keep = np.ones(T, bool)
    for _, a, b, _ in owned:
        keep[a:b] = False
    return keep


def dirty(pool, owned, fresh):
    """Slots that no sequence reads hold NaN: nothing of them may reach a result."""
    pool = pool.copy()
    read = {v for s, _, _, v in owned if not fresh[s]}
    for v in range(len(pool)):
        if v not in read:
            pool[v] = np.nan
    return pool


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D,view", [(1, False), (37, True), (64, False), (264, False), (520, True)])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_tokens_conv(name, D, view, W, dtype):
    r = gen(D + W)
    start, slot, fresh, slots = sequences(LENGTHS[name], D + W, before=2, empty=name != "one")
    T = int(start[-1]) + 3      # rows before the first sequence and behind the last one
    owned = R.owners(T, len(slot), slots, start, slot)
    rest = unowned(T, owned)
    x = tok_rows(T, D, dtype, r, view, rest)
    w, bias = dev(r.normal(size=(D, W)) / W), dev(r.normal(size=D))
    pool = dev(dirty(r.normal(size=(slots, D, W - 1)), owned, fresh), dtype)
    y = dev(r.normal(size=(T, D)), dtype)
    ref, err, pref = R.tokens_conv(f64(x), f64(w), f64(bias), True, f64(pool), start, slot, fresh, f64(y))
    y0, p0 = y.clone(), pool.clone()
    ssm.tokens_conv(x=x, w=w, bias=bias, silu=True, pool=pool, seq_start=torch.from_numpy(start).to(DEV),
                    slot=torch.from_numpy(slot).to(DEV), fresh=torch.from_numpy(fresh).to(DEV), out={"y": y})
    R.check("y", y, ref, err, dtype)
    R.check("pool", pool, pref, 0 * np.nan_to_num(pref), dtype)
    assert torch.equal(y[torch.from_numpy(rest).to(DEV)], y0[torch.from_numpy(rest).to(DEV)])
    idle = [v for v in range(slots) if v not in {o[3] for o in owned}]
    assert torch.equal(pool[idle].nan_to_num(), p0[idle].nan_to_num())


def scan_inputs(T, D, N, dtype, r, view=False, gate=True, poison=None):
    poison = np.zeros(T, bool) if poison is None else poison
    t = dict(delta=tok_rows(T, D, dtype, r, view, poison), x=tok_rows(T, D, dtype, r, view, poison))
    proj = r.normal(size=(T, 2 * N + 5))
    proj[poison] = np.nan
    proj = dev(proj, dtype)
    t["Bm"], t["C"] = proj[:, 5:5 + N], proj[:, 5 + N:]
    t["A"] = dev(-r.uniform(0.2, 8, (D, N)))
    t["delta_bias"] = dev(r.uniform(-5, 0.5, D))
    t["z"] = tok_rows(T, D, dtype, r, view, poison) if gate else None
    t["skip"] = dev(r.normal(size=D)) if gate else None
    return t


def scan_ref(t, softplus, pool, start, slot, fresh, y):
    return R.tokens_scan(f64(t["delta"]), f64(t["x"]), f64(t["A"]), f64(t["Bm"]), f64(t["C"]), f64(t["skip"]),
                         f64(t["z"]), f64(t["delta_bias"]), softplus, f64(pool), start, slot, fresh, f64(y))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,N,view", [(1, 1, False), (37, 16, True), (64, 16, False), (130, 7, False), (20, 8, True),
                                      (64, 4, False), (192, 16, True)])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_tokens_scan(name, D, N, view, dtype):
    r = gen(D + N)
    start, slot, fresh, slots = sequences(LENGTHS[name], D + N, before=2, empty=name not in ("one", "long"))
    T = int(start[-1]) + 3
    owned = R.owners(T, len(slot), slots, start, slot)
    rest = unowned(T, owned)
    t = scan_inputs(T, D, N, dtype, r, view, poison=rest)
    pool = dev(dirty(r.normal(size=(slots, D, N)), owned, fresh))
    y = dev(r.normal(size=(T, D)), dtype)
    ref, err, pref, perr = scan_ref(t, True, pool, start, slot, fresh, y)
    y0, p0 = y.clone(), pool.clone()
    ssm.tokens_scan(**t, delta_softplus=True, pool=pool, seq_start=torch.from_numpy(start).to(DEV),
                    slot=torch.from_numpy(slot).to(DEV), fresh=torch.from_numpy(fresh).to(DEV), out={"y": y})
    R.check("y", y, ref, err, dtype)
    R.check("pool", pool, pref, np.nan_to_num(perr), "f32")
    assert torch.equal(y[torch.from_numpy(rest).to(DEV)], y0[torch.from_numpy(rest).to(DEV)])
    idle = [v for v in range(slots) if v not in {o[3] for o in owned}]
    assert torch.equal(pool[idle].nan_to_num(), p0[idle].nan_to_num())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate,softplus", [(False, False), (False, True), (True, False)])
def test_tokens_scan_without_gate_or_transform(gate, softplus, dtype):
    r = gen(7)
    T, D, N = 75, 70, 16
    t = scan_inputs(T, D, N, dtype, r, gate=gate)
    t["delta"] = dev(r.uniform(0.001, 0.2, (T, D)), dtype)
    t["delta_bias"] = None
    pool = dev(r.normal(size=(2, D, N)))
    start = np.array([0, 40, T], np.int32)
    y = torch.zeros(T, D, dtype=DT[dtype], device=DEV)
    ref, err, pref, perr = scan_ref(t, softplus, pool, start, None, None, y)
    got = ssm.tokens_scan(**t, delta_softplus=softplus, pool=pool, seq_start=torch.from_numpy(start).to(DEV))
    R.check("y", got["y"], ref, err, dtype)
    R.check("pool", pool, pref, perr, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S,D,N,W", [(1, 1, 1, 2), (1, 64, 16, 4), (7, 37, 5, 3), (70, 72, 16, 4), (33, 264, 8, 2),
                                     (130, 40, 16, 4), (9, 40, 12, 4), (5, 300, 4, 3), (3, 513, 8, 2)])
def test_steps(S, D, N, W, dtype):
    """The step forms: one row a sequence, with empty places and a slot named twice."""
    r = gen(S + D)
    slot = r.permutation(S + 4)[:S].astype(np.int32)
    if S > 5:
        slot[3] = -1
        slot[S - 1] = slot[1]       # an earlier sequence has it
        slot[4] = S + 4             # outside the pool
    fresh = r.random(S) < 0.3
    owned = R.owners(S, S, S + 4, None, slot)
    ti = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    x, w, bias = tok_rows(S, D, dtype, r, True, []), dev(r.normal(size=(D, W))), dev(r.normal(size=D))
    pool = dev(dirty(r.normal(size=(S + 4, D, W - 1)), owned, fresh), dtype)
    y = dev(r.normal(size=(S, D)), dtype)
    ref, err, pref = R.tokens_conv(f64(x), f64(w), f64(bias), True, f64(pool), None, slot, fresh, f64(y))
    ssm.tokens_conv(x=x, w=w, bias=bias, silu=True, pool=pool, slot=ti(slot), fresh=ti(fresh), out={"y": y})
    R.check("conv y", y, ref, err, dtype)
    R.check("conv pool", pool, pref, 0 * np.nan_to_num(pref), dtype)
    t = scan_inputs(S, D, N, dtype, r, view=True)
    pool = dev(dirty(r.normal(size=(S + 4, D, N)), owned, fresh))
    y = dev(r.normal(size=(S, D)), dtype)
    ref, err, pref, perr = scan_ref(t, True, pool, None, slot, fresh, y)
    ssm.tokens_scan(**t, delta_softplus=True, pool=pool, slot=ti(slot), fresh=ti(fresh), out={"y": y})
    R.check("scan y", y, ref, err, dtype)
    R.check("scan pool", pool, pref, np.nan_to_num(perr), "f32")


def test_thousands_of_sequences():
    """More sequences than one round of the search through seq_start tells apart."""
    r = gen(61)
    D, N, W, S = 24, 5, 3, 5003
    start = np.concatenate([[0], np.cumsum(r.integers(0, 3, S))]).astype(np.int32)
    T = int(start[-1])
    slot = r.permutation(S).astype(np.int32)
    slot[17::100] = -1
    slot[4000] = slot[3]        # an earlier sequence has it
    fresh = r.random(S) < 0.5
    at = dict(seq_start=torch.from_numpy(start).to(DEV), slot=torch.from_numpy(slot).to(DEV),
              fresh=torch.from_numpy(fresh).to(DEV))
    x, w = tok_rows(T, D, "f32", r, False, []), dev(r.normal(size=(D, W)))
    pool, y = dev(r.normal(size=(S, D, W - 1))), dev(r.normal(size=(T, D)))
    ref, err, pref = R.tokens_conv(f64(x), f64(w), None, False, f64(pool), start, slot, fresh, f64(y))
    ssm.tokens_conv(x=x, w=w, pool=pool, out={"y": y}, **at)
    R.check("conv y", y, ref, err, "f32")
    R.check("conv pool", pool, pref, 0 * pref, "f32")
    t = scan_inputs(T, D, N, "f32", r)
    pool, y = dev(r.normal(size=(S, D, N))), dev(r.normal(size=(T, D)))
    ref, err, pref, perr = scan_ref(t, True, pool, start, slot, fresh, y)
    ssm.tokens_scan(**t, delta_softplus=True, pool=pool, out={"y": y}, **at)
    R.check("scan y", y, ref, err, "f32")
    R.check("scan pool", pool, pref, perr, "f32")


@pytest.mark.parametrize("many", [False, True])
def test_lists_that_do_not_ascend_stay_inside_the_buffers(many):
    """seq_start, slot and fresh are not checked on the host: whatever they hold, nothing outside the rows of y and the
    slots of the pool is written (what the rows then hold is unspecified)."""
    r = gen(62)
    D, N, W, T, S = 40, 16, 4, 300, 90 if many else 6
    big = np.iinfo(np.int32)
    starts = [[250, 0, 10, 290, 20, 300, 0], [500, 600, -7, 40, big.max, big.min, 299], [big.max] * 7,
              [-3, 200, 100, 299, 298, 10, 1000], [299, 300, 301, 302, 303, 304, 305], [300, 250, 200, 150, 100, 50, 0]]
    if many:
        starts = [r.integers(-50, 400, S + 1) for _ in range(4)] + [np.arange(S, -1, -1) * 4]
    rows = torch.full((T + 2, D + 9), 7.0, device=DEV)
    pools = [torch.full((S + 2, D, k), 7.0, device=DEV) for k in (W - 1, N)]
    w, x = dev(r.normal(size=(D, W))), tok_rows(T, D, "f32", r, True, [])
    t = scan_inputs(T, D, N, "f32", r, view=True)
    for i, st in enumerate(starts):
        slot = r.integers(0, S, S)
        slot[i % S] = (big.max, big.min, S, -1)[i % 4]
        at = dict(seq_start=torch.tensor(np.asarray(st), dtype=torch.int32, device=DEV),
                  slot=torch.tensor(slot, dtype=torch.int32, device=DEV),
                  fresh=torch.tensor(r.integers(0, 256, S), dtype=torch.uint8, device=DEV))
        y = rows[1:T + 1, 4:4 + D]
        ssm.tokens_conv(x=x, w=w, pool=pools[0][1:-1], out={"y": y}, **at)
        ssm.tokens_scan(**t, delta_softplus=True, pool=pools[1][1:-1], out={"y": y}, **at)
        torch.cuda.synchronize()
        assert (rows[0] == 7).all() and (rows[-1] == 7).all() and (rows[:, :4] == 7).all() and (rows[:, 4 + D:] == 7).all()
        assert all((p[0] == 7).all() and (p[-1] == 7).all() for p in pools)


def test_offsets_past_32_bits():
    """Rows and slots of the widest strides, and batch rows 2^32 elements apart: as the same tensors laid out densely."""
    r = gen(63)
    D, N, W, T, S = 24, 16, 4, 70, 3
    wide, wide_out = (torch.empty(T * 2**26, dtype=torch.bfloat16, device=DEV) for _ in range(2))

    def spread(v, at):
        o = wide.as_strided(v.shape, (2**26 - 1, 1), at)
        o.copy_(v)
        return o

    t = scan_inputs(T, D, N, "bf16", r)
    far = {k: spread(t[k], 100 * i) for i, k in enumerate(("delta", "x", "z", "Bm", "C"))}
    w = dev(r.normal(size=(D, W)))
    at = dict(seq_start=torch.tensor([0, 33, 34, T], dtype=torch.int32, device=DEV),
              slot=torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV))
    for k, inner, dt in (("c", W - 1, torch.bfloat16), ("s", N, torch.float32)):
        first = torch.randn(S, D, inner, device=DEV).to(dt)
        base = torch.empty(2 * (2**30 + 4) + D * inner, dtype=dt, device=DEV)
        res = []
        for f in (False, True):
            for step in (False, True):
                pool = base.as_strided(first.shape, (2**30 + 4, inner, 1)) if f else torch.empty_like(first)
                pool.copy_(first)
                a = {**t, **far} if f else t
                a = {n: v[:S] if step and n in far else v for n, v in a.items()}
                on = dict(slot=at["slot"]) if step else at
                out = {"y": wide_out.as_strided((S if step else T, D), (2**26 - 1, 1), 900)} if f else {}
                y = (ssm.tokens_conv(x=a["x"], w=w, pool=pool, out=out, **on) if k == "c" else
                     ssm.tokens_scan(**a, delta_softplus=True, pool=pool, out=out, **on))["y"]
                res += [y.clone(), pool.clone()]
        for p, q in zip(res[:4], res[4:]):
            assert torch.equal(p, q), k
        del base, pool
    x = dev(r.normal(size=(2, 3, 700)), "bf16")
    gy = dev(r.normal(size=(2, 3, 700)), "bf16")
    fx, fg, fo = (v.as_strided(x.shape, (2**32, 2**20, 1), i) for v, i in ((wide, 0), (wide, 5000), (wide_out, 3)))
    fx.copy_(x)
    fg.copy_(gy)
    par = dict(w=w[:3], silu=True)
    assert torch.equal(ssm.conv_fwd(x=fx, out={"y": fo}, **par)["y"], ssm.conv_fwd(x=x, **par)["y"])
    p, q = ssm.conv_bwd(x=x, gy=gy, **par), ssm.conv_bwd(x=fx, gy=fg, out={"gx": fo}, **par)
    assert all(torch.equal(p[k], q[k]) for k in p)
    p, q = ssm.ckpt8_pack(x), ssm.ckpt8_pack(fx)
    assert all(torch.equal(p[k], q[k]) for k in p)
    assert torch.equal(ssm.ckpt8_unpack(**p, dtype=torch.bfloat16, out=fo), ssm.ckpt8_unpack(**p, dtype=torch.bfloat16))


def test_pool_of_a_layer_among_others():
    """Pools that are one layer's slice of all layers' (slot stride wider than a slot)."""
    r = gen(12)
    S, D, N = 6, 40, 16
    wide = dev(r.normal(size=(S, 3, D, N)))
    before = wide.clone()
    t = scan_inputs(S, D, N, "f32", r)
    one = wide[:, 1].contiguous()
    ssm.tokens_scan(**t, pool=one)
    ssm.tokens_scan(**t, pool=wide[:, 1])
    assert torch.equal(wide[:, 1], one) and torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, 2], before[:, 2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_then_tokens_as_one_layer(dtype):
    """A layer's serving path: prompts through convolution and scan, then tokens one by one; against the training
    kernels over the whole sequences."""
    r = gen(90)
    D, N, W, steps = 72, 16, 4, 5
    lengths = [37, 1, 90, 3]
    S = len(lengths)
    full = [n + steps for n in lengths]
    w, bias = dev(r.normal(size=(D, W)) / 2), dev(r.normal(size=D))
    A, skip, dbias = dev(-r.uniform(0.5, 4, (D, N))), dev(r.normal(size=D)), dev(r.uniform(-4, -1, D))
    xs = [dev(r.normal(size=(n, D)), dtype) for n in full]
    dl = [dev(r.normal(size=(n, D)), dtype) for n in full]
    bc = [dev(r.normal(size=(n, 2 * N)), dtype) for n in full]
    cpool, spool = torch.zeros(S, D, W - 1, dtype=DT[dtype], device=DEV), torch.zeros(S, D, N, device=DEV)
    slot = torch.tensor([2, 0, 3, 1], dtype=torch.int32, device=DEV)
    par = dict(A=A, skip=skip, delta_bias=dbias, delta_softplus=True, pool=spool, slot=slot)

    def rows(parts, lo, hi):
        return torch.cat([p[lo(n):hi(n)] for p, n in zip(parts, lengths)])

    start = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
    got = [[] for _ in range(S)]
    at = dict(seq_start=start, fresh=torch.ones(S, dtype=torch.bool, device=DEV))
    for k in range(steps + 1):
        lo, hi = (lambda n: 0, lambda n: n) if k == 0 else (lambda n: n + k - 1, lambda n: n + k)
        u = ssm.tokens_conv(x=rows(xs, lo, hi), w=w, bias=bias, silu=True, pool=cpool, slot=slot, **at)["y"]
        b = rows(bc, lo, hi)
        o = ssm.tokens_scan(delta=rows(dl, lo, hi), x=u, Bm=b[:, :N], C=b[:, N:], **par, **at)["y"]
        for i, part in enumerate(torch.split(o, lengths if k == 0 else [1] * S)):
            got[i].append(part)
        at = {}
    for i in range(S):
        x = xs[i].T[None].contiguous()
        u = ssm.conv_fwd(x=x, w=w, bias=bias, silu=True)["y"]
        f = ssm.scan_fwd(ssm.SSM_REAL_SELECTIVE, want_h_last=True, delta=dl[i].T[None].contiguous(), x=u, A=A,
                         Bm=bc[i][None, :, :N].contiguous(), C=bc[i][None, :, N:].contiguous(), delta_bias=dbias,
                         delta_softplus=True)
        ref = f64(f["y"])[0].T + f64(skip) * f64(u)[0].T
        # u is equal bit for bit; the training kernel rounds y to the stream's type before the skip is added here
        mag = np.abs(ref) + np.abs(f64(f["y"])[0].T)
        lim = 2 * R.HALF[dtype] * mag + 2e-5 * np.abs(mag).max()
        assert (np.abs(f64(torch.cat(got[i])) - ref) <= lim).all()
        v = int(slot[i])
        assert torch.equal(cpool[v], xs[i][-3:].T)
        h = f64(f["h_last"])[0]
        assert (np.abs(f64(spool[v]) - h) <= 1e-5 * np.abs(h).max()).all()


def test_layer_backward_from_checkpoints():
    """Convolution and scan of a layer with the convolution's input kept in 8 bits: the backward pass recomputes the
    scan's input from the checkpoint; against the float64 chain on the values the checkpoint stands for."""
    r = gen(17)
    B, D, L, N, W = 2, 16, 200, 16, 4
    x, w, bias = dev(r.normal(size=(B, D, L))), dev(r.normal(size=(D, W)) / 2), dev(r.normal(size=D) * 0.2)
    t = dict(delta=dev(r.uniform(0.01, 0.2, (B, D, L))), A=dev(-r.uniform(0.5, 4, (D, N))),
             Bm=dev(r.normal(size=(B, L, N))), C=dev(r.normal(size=(B, L, N))))
    gy = dev(r.normal(size=(B, D, L)))
    par = dict(w=w, bias=bias, silu=True)
    kept = ssm.conv_fwd(x=x, want_ckpt8=True, **par)
    c8 = (kept["x8"], kept["x8_scale"])
    u = ssm.conv_fwd(ckpt8=c8, dtype=torch.float32, **par)["y"]
    f = ssm.scan_fwd(ssm.SSM_REAL_SELECTIVE, want_ckpt=True, x=u, **t)
    g = ssm.scan_bwd(ssm.SSM_REAL_SELECTIVE, gy=gy, ckpt=f["ckpt"], x=u, **t)
    got = ssm.conv_bwd(gy=g["gx"], ckpt8=c8, **par)
    x64 = R.unpack(c8[0].cpu().numpy(), c8[1].cpu().numpy()).astype(np.float64)
    u64, uerr, _ = R.conv_fwd(x64, f64(w), f64(bias), None, True)
    R.check("scan input", u, u64, uerr, "f32")
    ref = R.conv_bwd(x64, f64(w), f64(bias), None, True, f64(g["gx"]), None)
    for k in ("gx", "gw", "gbias"):
        R.check(k, got[k], *ref[k], "f32")


def test_streams_and_graphs():
    """Calls on a stream of their own, and captured calls replayed with other inputs, eager work and waits between them:
    every replay equals the eager call bit for bit."""
    r = gen(50)
    D, N, W, S = 96, 16, 4, 6
    start = torch.tensor([0, 30, 31, 31, 90, 200, 333], dtype=torch.int32, device=DEV)
    T = 333
    slot = torch.tensor([3, 1, 2, 7, 5, -1], dtype=torch.int32, device=DEV)
    w, bias = dev(r.normal(size=(D, W))), dev(r.normal(size=D))
    t = scan_inputs(T, D, N, "bf16", r)
    xc, gyc, _ = dev(r.normal(size=(2, D, 130))), dev(r.normal(size=(2, D, 130))), None
    cpool, spool = dev(r.normal(size=(8, D, W - 1)), "bf16"), dev(r.normal(size=(8, D, N)))
    keep = [v.clone() for v in (cpool, spool)]

    def run():
        o = {}
        cpool.copy_(keep[0])
        spool.copy_(keep[1])
        o["c"] = ssm.tokens_conv(x=t["x"], w=w, bias=bias, silu=True, pool=cpool, seq_start=start, slot=slot,
                                 out={"y": torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)})["y"]
        o["s"] = ssm.tokens_scan(**{**t, "x": o["c"]}, delta_softplus=True, pool=spool, seq_start=start, slot=slot,
                                 out={"y": torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)})["y"]
        o["s1"] = ssm.tokens_scan(**{k: v[:6] if k in ("delta", "x", "z", "Bm", "C") else v for k, v in t.items()},
                                  pool=spool, slot=slot, out={"y": torch.zeros(6, D, dtype=torch.bfloat16, device=DEV)})["y"]
        f = ssm.conv_fwd(x=xc, w=w, bias=bias, silu=True, want_ckpt8=True)
        o.update({k: v for k, v in f.items()})
        o.update(ssm.conv_bwd(gy=gyc, ckpt8=(f["x8"], f["x8_scale"]), w=w, bias=bias, silu=True))
        o["cpool"], o["spool"] = cpool.clone(), spool.clone()
        return o

    ref = run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        own = run()
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k], own[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run()
    for i in range(4):
        xc.copy_(dev(r.normal(size=(2, D, 130))))
        t["x"].copy_(dev(r.normal(size=(T, D)), "bf16"))
        keep[1].copy_(dev(r.normal(size=(8, D, N))))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in cap.items()}
        eager = run()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(eager[k], got[k]), (i, k)


# ---------------------------------------------------------------------------
# the binding's two ways into the library
# ---------------------------------------------------------------------------
def layer_calls(seed):
    """Every function of this file once, with plain tensors; {name: outputs}."""
    r = gen(seed)
    D, N, W = 72, 16, 4
    t, gy, glast = conv_inputs(2, 9, 1100, W, "bf16", True, seed)
    par = dict(w=t["w"], bias=t["bias"], init=t["init"], silu=True)
    o = {}

    def keep(name, d):
        o.update({f"{name} {k}": v for k, v in (d.items() if isinstance(d, dict) else [("y", d)])})
        return d

    f = keep("fwd", ssm.conv_fwd(x=t["x"], want_last=True, want_ckpt8=True, **par))
    keep("fwd only last", ssm.conv_fwd(x=t["x"], want_y=False, want_last=True, **par))
    keep("bwd", ssm.conv_bwd(gy=gy, glast=glast, x=t["x"], **par))
    keep("bwd8", ssm.conv_bwd(gy=gy, ckpt8=(f["x8"], f["x8_scale"]), want=("gw", "gx"), **par))
    keep("pack", ssm.ckpt8_pack(t["x"]))
    keep("unpack", ssm.ckpt8_unpack(f["x8"], f["x8_scale"], dtype=torch.bfloat16))
    keep("unpack32", ssm.ckpt8_unpack(f["x8"], f["x8_scale"]))
    start, slot, fresh, slots = sequences([3, 0, 41, 1, 9], seed, empty=False)
    T = int(start[-1])
    at = dict(seq_start=torch.from_numpy(start).to(DEV), slot=torch.from_numpy(slot).to(DEV),
              fresh=torch.from_numpy(fresh).to(DEV))
    cpool, spool = dev(r.normal(size=(slots, D, W - 1)), "bf16"), dev(r.normal(size=(slots, D, N)))
    x = tok_rows(T, D, "bf16", r, True, [])
    s = scan_inputs(T, D, N, "bf16", r, view=True)
    w, b = dev(r.normal(size=(D, W))), dev(r.normal(size=D))
    y = torch.zeros(T, D + 8, dtype=torch.bfloat16, device=DEV)[:, :D]
    keep("tconv", ssm.tokens_conv(x=x, w=w, bias=b, silu=True, pool=cpool, **at))
    got = ssm.tokens_conv(x=x, w=w, pool=cpool, out={"y": y}, **at)
    assert got["y"] is y
    keep("tconv2", got)
    keep("tscan", ssm.tokens_scan(**s, delta_softplus=True, pool=spool, **at))
    step = {k: v[:5] if k in ("delta", "x", "z", "Bm", "C") else v for k, v in s.items()}
    keep("tstep", ssm.tokens_scan(**{**step, "z": None, "skip": None}, pool=spool, slot=at["slot"]))
    keep("pools", {"c": cpool, "s": spool})
    torch.cuda.synchronize()
    return o


def test_native_calls_are_the_bindings():
    """Without an installed allocator plain calls go through the native module: the same keys and the same bits."""
    a = layer_calls(3)
    ssm.set_allocator(None)
    from selective_state_space_chunked_amd import binding
    made = []
    orig = binding._done

    def count(r):
        made.append(r is not NotImplemented)
        return orig(r)

    binding._done = count
    try:
        b = layer_calls(3)
    finally:
        binding._done = orig
    assert made and all(made)
    assert a.keys() == b.keys()
    for k in a:
        assert a[k].dtype == b[k].dtype and a[k].shape == b[k].shape and torch.equal(a[k], b[k]), k


def test_wanted_gradients_from_an_iterator():
    t, gy, glast = conv_inputs(1, 4, 40, 4, "f32", True, 64)
    par = dict(gy=gy, glast=glast, x=t["x"], w=t["w"], bias=t["bias"], init=t["init"])
    every, some = ssm.conv_bwd(**par), ssm.conv_bwd(want=(k for k in ("gw", "ginit")), **par)
    assert set(some) == {"gw", "ginit"} and all(torch.equal(some[k], every[k]) for k in some)


def test_native_calls_refuse_as_the_binding():
    """Arguments the native module leaves alone raise the binding's errors; those the library refuses, the library's."""
    ssm.set_allocator(None)
    x, w = torch.zeros(2, 3, 10, device=DEV), torch.zeros(3, 4, device=DEV)
    rows, pool = torch.zeros(6, 3, device=DEV), torch.zeros(4, 3, 3, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    for f, kw, exc in ((ssm.conv_fwd, dict(x=x, w=torch.zeros(3, 5, device=DEV)), ssm.binding.SSMError),
                       (ssm.conv_fwd, dict(x=x, w=torch.zeros(2, 4, device=DEV)), ValueError),
                       (ssm.conv_fwd, dict(x=x.double(), w=w), TypeError),
                       (ssm.conv_fwd, dict(x=x, w=w.cpu()), ValueError),
                       (ssm.conv_bwd, dict(gy=x[..., :9], x=x, w=w), ValueError),
                       (ssm.conv_bwd, dict(gy=x, x=x, w=w, want=("gz",)), ValueError),
                       (ssm.tokens_conv, dict(x=rows, w=w, pool=pool), ssm.binding.SSMError),      # 6 rows, 4 slots
                       (ssm.tokens_conv, dict(x=rows, w=w, pool=pool.bfloat16(), slot=torch.zeros(6, **i32)), TypeError),
                       (ssm.tokens_conv, dict(x=rows, w=w, pool=pool, slot=torch.zeros(5, **i32)), ValueError),
                       (ssm.tokens_scan, dict(delta=rows, x=rows, A=torch.zeros(3, 17, device=DEV),
                                              Bm=torch.zeros(6, 17, device=DEV), C=torch.zeros(6, 17, device=DEV),
                                              pool=torch.zeros(6, 3, 17, device=DEV)), ssm.binding.SSMError),
                       (ssm.tokens_scan, dict(delta=rows, x=rows, A=torch.zeros(3, 4, device=DEV),
                                              Bm=torch.zeros(6, 5, device=DEV), C=torch.zeros(6, 4, device=DEV),
                                              pool=torch.zeros(6, 3, 4, device=DEV)), ValueError),
                       (ssm.tokens_conv, dict(x=rows, w=w, pool=pool, slot=torch.zeros(6, **i32),
                                              out={"y": rows}), ssm.binding.SSMError)):            # y over x
        with pytest.raises(exc):
            f(**kw)


# ---------------------------------------------------------------------------
# ends of the ranges
# ---------------------------------------------------------------------------
def largest_inputs(B, D, L, dtype, top, seed):
    """A stream of every size up to `top`, some elements +-top and some 0; weights and gradients that keep sums finite."""
    r = gen(seed)
    x = r.uniform(-1, 1, (B, D, L)) * top
    x[..., ::9] = top
    x[..., 5::9] = -top
    x[..., 3::7] = 0.0
    w = r.uniform(0.5, 1, (D, 4)) * r.choice([-1, 1], (D, 4)) * 2.0 ** -124     # four taps: |p| below 70
    t = dict(x=dev(x, dtype), w=dev(w), bias=dev(r.normal(size=D)), init=None)
    return t, dev(r.normal(size=(B, D, L)) * 2.0 ** -12, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,L", [(2, 3, 131), (1, 5, 1099), (2, 5, 1104), (1, 3, 513)])
def test_ckpt8_of_the_largest_values(B, D, L, dtype):
    """Blocks up to the largest value whose 127 scales are finite: the bytes times their scale, rounded once, in every
    reader of a checkpoint (runs, rows' ends, whole tiles and what lies beside them)."""
    top = float(torch.finfo(torch.bfloat16).max) if dtype == "bf16" else (2 - 2.0 ** -22) * 2.0 ** 127
    t, gy = largest_inputs(B, D, L, dtype, top, L)
    f = ssm.conv_fwd(x=t["x"], w=t["w"], bias=t["bias"], silu=True, want_ckpt8=True)
    q, s = R.pack(t["x"].float().cpu().numpy())
    assert np.array_equal(f["x8"].cpu().numpy(), q) and np.array_equal(f["x8_scale"].cpu().numpy(), s)
    kept = R.unpack(q, s)
    assert np.isfinite(kept).all()
    c8 = (f["x8"], f["x8_scale"])
    assert np.array_equal(ssm.ckpt8_unpack(*c8).cpu().numpy(), kept)
    assert torch.equal(ssm.ckpt8_unpack(*c8, dtype=torch.bfloat16).cpu(), torch.from_numpy(kept).bfloat16())
    conv_check(t, gy, None, True, dtype, x64=kept.astype(np.float64), ckpt8=c8)


def test_ckpt8_of_the_largest_float():
    """127 times the scale rounded from it would be infinite: the scale is one step less, and every element finite."""
    top = np.finfo(np.float32).max
    t, gy = largest_inputs(2, 3, 1099, "f32", float(top), 5)
    f = ssm.conv_fwd(x=t["x"], w=t["w"], bias=t["bias"], silu=True, want_ckpt8=True)
    q, s = R.pack(t["x"].cpu().numpy())
    s = np.minimum(s, np.nextafter(top / np.float32(127), np.float32(0)))
    assert np.array_equal(f["x8"].cpu().numpy(), q) and np.array_equal(f["x8_scale"].cpu().numpy(), s)
    kept = R.unpack(q, s)
    assert np.isfinite(kept).all() and np.abs(kept).max() == np.nextafter(top, np.float32(0))
    c8 = (f["x8"], f["x8_scale"])
    assert np.array_equal(ssm.ckpt8_unpack(*c8).cpu().numpy(), kept)
    conv_check(t, gy, None, True, "f32", x64=kept.astype(np.float64), ckpt8=c8)


def test_native_calls_without_memory():
    """No memory for an output: torch's OutOfMemoryError, as from the binding's own path, and the next call is fine."""
    ssm.set_allocator(None)
    x8, scale = torch.ones(1, 64, 1 << 20, dtype=torch.int8, device=DEV), torch.ones(1, 64, 1 << 14, device=DEV)
    w, gy = torch.ones(64, 4, device=DEV), torch.ones(1, 64, 1 << 20, device=DEV)
    ref = ssm.ckpt8_unpack(x8[:, :1].contiguous(), scale[:, :1].contiguous())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(
        (torch.cuda.memory_reserved() + (64 << 20)) / torch.cuda.get_device_properties(0).total_memory)
    try:
        for call in (lambda: ssm.ckpt8_unpack(x8, scale), lambda: ssm.conv_fwd(x=gy, w=w),
                     lambda: ssm.conv_bwd(gy=gy, ckpt8=(x8, scale), w=w)):
            with pytest.raises(torch.OutOfMemoryError):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.equal(ssm.ckpt8_unpack(x8, scale)[:, :1], ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_last_tokens_of_long_rows(dtype):
    """The last token of each of two long sequences, a slice whose rows are 2^26 elements apart, through the step forms
    and as prompts of one row: as the same rows laid out densely."""
    r = gen(71)
    D, N, W, S = 2048, 16, 4, 2
    hidden = torch.zeros(S, 2 ** 15, D, dtype=DT[dtype], device=DEV)
    t = scan_inputs(S, D, N, dtype, r)
    hidden[:, -1] = t["x"]
    far = hidden[:, -1]
    assert far.stride() == (2 ** 26, 1)
    w, one = dev(r.normal(size=(D, W))), torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    cpool, spool = dev(r.normal(size=(S, D, W - 1)), dtype), dev(r.normal(size=(S, D, N)))
    rows = ("delta", "x", "z", "Bm", "C")
    for n, at in ((S, {}), (1, dict(seq_start=one)), (1, {})):
        cut = {k: v[:n] if k in rows else v for k, v in t.items()}
        res = []
        for x in (far[:n], t["x"][:n]):
            c, s = cpool[:n].clone(), spool[:n].clone()
            a = {k: x if k in ("delta", "x", "z") else v for k, v in cut.items()}
            res.append([ssm.tokens_conv(x=x, w=w, silu=True, pool=c, **at)["y"],
                        ssm.tokens_scan(**a, delta_softplus=True, pool=s, **at)["y"], c, s])
        assert all(torch.equal(p, q) for p, q in zip(*res))
    c1, c2 = cpool.clone(), cpool.clone()
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    p, q = (ssm.tokens_conv(x=x, w=w, pool=c, seq_start=start)["y"] for x, c in ((far, c1), (t["x"], c2)))
    assert torch.equal(p, q) and torch.equal(c1, c2)
    with pytest.raises(ssm.binding.SSMError):      # the scan of prompts ends at 2^26
        ssm.tokens_scan(**{**t, "x": far}, pool=spool.clone(), seq_start=start)


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("N", range(1, 17))
def test_tokens_scan_of_every_state_size(N, layer):
    """Each state size has a kernel and a layout of its own: prompts over more ranges than a wave composes by itself, with
    skip, gate and softplus and without, and the same states in steps."""
    r = gen(100 + N)
    D, lengths = 70, [5, 1, 0, 17, 390, 64, 2]
    start, slot, fresh, slots = sequences(lengths, N, empty=False)
    T = int(start[-1])
    t = scan_inputs(T, D, N, "bf16" if N % 2 else "f32", r, view=True, gate=layer)
    dtype = "bf16" if N % 2 else "f32"
    if not layer:
        t["delta"], t["delta_bias"] = dev(r.uniform(0.001, 0.2, (T, D)), dtype), None
    owned = R.owners(T, len(slot), slots, start, slot)
    pool, y = dev(dirty(r.normal(size=(slots, D, N)), owned, fresh)), torch.zeros(T, D, dtype=DT[dtype], device=DEV)
    ref, err, pref, perr = scan_ref(t, layer, pool, start, slot, fresh, y)
    got = ssm.tokens_scan(**t, delta_softplus=layer, pool=pool, seq_start=torch.from_numpy(start).to(DEV),
                          slot=torch.from_numpy(slot).to(DEV), fresh=torch.from_numpy(fresh).to(DEV), out={"y": y})
    R.check("y", got["y"], ref, err, dtype)
    R.check("pool", pool, pref, np.nan_to_num(perr), "f32")
    S = 5
    step = {k: v[:S] if k in ("delta", "x", "z", "Bm", "C") and v is not None else v for k, v in t.items()}
    pool = dev(r.normal(size=(S, D, N)))
    ref, err, pref, perr = scan_ref(step, layer, pool, None, None, None, y[:S])
    got = ssm.tokens_scan(**step, delta_softplus=layer, pool=pool)
    R.check("step y", got["y"], ref, err, dtype)
    R.check("step pool", pool, pref, perr, "f32")


def test_native_calls_in_a_graph():
    """The native calls allocate outputs and workspaces in a captured graph's own memory: replays with other inputs, eager
    calls and waits between them, equal the eager calls bit for bit."""
    ssm.set_allocator(None)
    r = gen(81)
    D, N, W, T = 72, 16, 4, 600
    t, gy, glast = conv_inputs(3, D, 1100, W, "bf16", True, 82)
    s = scan_inputs(T, D, N, "bf16", r, view=True)
    at = dict(seq_start=torch.tensor([0, 31, 31, 590, T], dtype=torch.int32, device=DEV),
              slot=torch.tensor([3, 0, 2, 1], dtype=torch.int32, device=DEV))
    pools = [dev(r.normal(size=(4, D, W - 1)), "bf16"), dev(r.normal(size=(4, D, N)))]
    keep = [p.clone() for p in pools]

    def run():
        for p, k in zip(pools, keep):
            p.copy_(k)
        o = dict(ssm.conv_fwd(x=t["x"], w=t["w"], bias=t["bias"], init=t["init"], silu=True, want_ckpt8=True))
        o.update(ssm.conv_bwd(gy=gy, glast=glast, ckpt8=(o["x8"], o["x8_scale"]), w=t["w"], bias=t["bias"],
                              init=t["init"], silu=True))
        o["back"] = ssm.ckpt8_unpack(o["x8"], o["x8_scale"], dtype=torch.bfloat16)
        o["c"] = ssm.tokens_conv(x=s["x"], w=t["w"], bias=t["bias"], silu=True, pool=pools[0], **at)["y"]
        o["s"] = ssm.tokens_scan(**{**s, "x": o["c"]}, delta_softplus=True, pool=pools[1], **at)["y"]
        o["pools"] = torch.cat([p.float().flatten() for p in pools])
        return o

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run()
    for i in range(4):
        t["x"].copy_(dev(r.normal(size=t["x"].shape), "bf16"))
        s["x"].copy_(dev(r.normal(size=s["x"].shape), "bf16"))
        keep[1].copy_(dev(r.normal(size=keep[1].shape)))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in cap.items()}
        eager = run()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(eager[k], got[k]), (i, k)

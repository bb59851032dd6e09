"""The gated layer's operators on the GPU where their kernels take other ways than at the sizes of test_gpu_gated.py: rows of
several tiles, values that are not finite beside lanes without channels.  Which kernel a call runs is asked of the library's
diagnostics, so that a size whose kernel changes fails its test."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_chunked_amd as ssm
from selective_state_space_chunked_amd import binding

from . import _gated_ref as R
from . import _layer_ref as C
from .test_gpu_gated import DEV, DT, GATED_OUT, dev, f64, gated_inputs, gen, mm8_check, mm8_inputs, norm_check, norm_inputs

pytestmark = pytest.mark.gpu


def launched(f):
    """f's result and the names of the kernels its calls enqueued."""
    L, n, names = binding.lib(), ctypes.c_int(0), (ctypes.c_char_p * 64)()
    assert L.ssm_profile_begin(ctypes.c_int(64)) == 0
    try:
        r = f()
    finally:
        rc = L.ssm_profile_end(ctypes.byref(n), (ctypes.c_float * 64)(), names, ctypes.c_int(64))
    assert rc == 0
    return r, [names[i].decode() for i in range(n.value)]


# ---------------------------------------------------------------------------
# gated recurrence
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,L,lanes", [(8, 8200, 299, 16), (8, 2051, 1100, 64), (5, 900, 4500, 256), (3, 40, 20011, 1024)])
def test_gated_rows_of_several_tiles(B, D, L, lanes, dtype):
    """Each number of lanes a row goes round its tiles three times, the last time with a part of one: states and mu are
    carried from tile to tile, in slow channels over all of the row.  Against the reference for some of the channels."""
    r = gen(B + L)
    t, gy, gl = gated_inputs(B, D, L, dtype, r)
    t["lam"][::2] -= 6.0
    f, names = launched(lambda: ssm.gated_fwd(want_h_last=True, want_ckpt=True, **t))
    assert names == [f"gated recurrence, {lanes} lanes a row"] and 2 * lanes * 8 < L < 3 * lanes * 8
    g, names = launched(lambda: ssm.gated_bwd(gy=gy, gh_last=gl, ckpt=f["ckpt"], **t))
    assert names[0] == f"gated recurrence backward, {lanes} lanes a row"
    some = sorted({0, 1, 2, 3, D // 2, D - 2, D - 1, *(int(v) for v in r.integers(0, D, 5))})
    v = [f64(t[k][some] if k in ("lam", "r_bias", "i_bias") else t[k][:, some]) for k in ("x", "r", "i", "lam", "r_bias", "i_bias")]
    v += [8.0, f64(t["h0"][:, some])]
    ref = {**R.gated_fwd(*v), **R.gated_bwd(*v, f64(gy[:, some]), f64(gl[:, some]))}
    for k, got in {"y": f["y"], "h_last": f["h_last"], **g}.items():
        R.check(k, got[some] if got.dim() == 1 else got[:, some], *ref[k], "f32" if k in GATED_OUT else dtype)
    again = ssm.gated_bwd(gy=gy, gh_last=gl, **t)   # the states formed again
    assert all(torch.equal(g[k], again[k]) for k in g)


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G,per", [(4, 24), (5, 3), (3, 65), (2, 520), (2, 519), (2, 2056), (2, 2501)])
def test_norm_non_finite_values_stay_in_their_group(G, per, dtype):
    """What is not finite in x, z or gy of one group of one row, or in w and bias of one channel, reaches that group's (that
    channel's group's) results and no other's: groups whose last lanes have no channels among them."""
    r = gen(G + per)
    T, width = 9, G * per
    t, gy = norm_inputs(T, width, dtype, r)
    ref = {**ssm.group_norm_fwd(groups=G, silu=True, **t), **ssm.group_norm_bwd(gy=gy, groups=G, silu=True, **t)}
    for name in ("x", "z", "gy", "w", "bias"):
        for at in (0, per, width - 1):
            for bad in (float("nan"), float("inf"), -float("inf")):
                u = {**t, "gy": gy}
                u[name] = u[name].clone()
                rows = slice(None) if name in ("w", "bias") else 5
                u[name][(at,) if name in ("w", "bias") else (5, at)] = bad
                g = u.pop("gy")
                got = {**ssm.group_norm_fwd(groups=G, silu=True, **u), **ssm.group_norm_bwd(gy=g, groups=G, silu=True, **u)}
                own = slice(at // per * per, (at // per + 1) * per)
                for k in ref:
                    keep = torch.ones_like(ref[k], dtype=torch.bool)
                    if k in ("gw", "gbias"):
                        keep[own] = False
                    else:
                        keep[rows, own] = False
                    assert torch.equal(got[k][keep], ref[k][keep]), (name, at, bad, k)


VECTOR, TWO, EIGHT = "a vector each", "two vectors each", "eight channels each"


@pytest.mark.parametrize("dtype,per,lanes,form", [
    ("bf16", 64, 64, VECTOR), ("f32", 64, 64, VECTOR), ("bf16", 520, 64, TWO), ("f32", 264, 64, TWO), ("bf16", 1032, 256, VECTOR),
    ("f32", 1020, 256, VECTOR), ("bf16", 2056, 256, TWO), ("f32", 1032, 256, TWO), ("bf16", 4104, 1024, VECTOR),
    ("f32", 2056, 1024, VECTOR), ("f32", 4100, 1024, TWO), ("bf16", 519, 256, EIGHT), ("f32", 519, 256, EIGHT),
    ("bf16", 2051, 1024, EIGHT), ("f32", 2501, 1024, EIGHT)])
def test_norm_teams_of_several_rows(dtype, per, lanes, form):
    """Every team of every kernel takes three rows and some a fourth: the row after is loaded meanwhile, the sums of a team
    of several waves go through the same places again, the parameters' gradients add up over a team's rows."""
    G = 3 if lanes == 64 else 1
    width = G * per
    # chunks of workgroups share the rows, as many as the backward keeps partial sums of
    chunks = binding._norm_bwd_bytes(binding._STREAM[torch.float32 if dtype == "f32" else torch.bfloat16], 1 << 20, width, G) // (8 * width)
    step = chunks * (8 if lanes == 64 else 1)
    T = 3 * step + step // 3 + 1
    t, gy = norm_inputs(T, width, dtype, gen(per))
    f, names = launched(lambda: ssm.group_norm_fwd(groups=G, silu=True, **t))
    assert names == [f"group norm, {lanes} lanes, {form}"]
    g, names = launched(lambda: ssm.group_norm_bwd(gy=gy, groups=G, silu=True, **t))
    assert names[0] == f"group norm backward, {lanes} lanes, {form}"
    ref = R.norm(f64(t["x"]), G, f64(t["w"]), f64(t["bias"]), 1e-5, True, f64(t["z"]), f64(gy))
    for k, v in {**f, **g}.items():
        R.check(k, v, *ref[k], "f32" if k in ("gw", "gbias") else dtype)


# ---------------------------------------------------------------------------
# products in 8-bit integers
# ---------------------------------------------------------------------------
def product(tile, whole):
    return "product in 8-bit integers, " + (f"tiles of {tile}" if tile else "few rows") + ("" if whole else ", through registers")


@pytest.mark.parametrize("T,K,N,tile,side", [
    (4096, 128, 4352, 256, 128), (4096, 336, 4352, 256, 128), (4096, 16, 4352, 256, 128), (4100, 384, 4300, 256, 128),
    (3800, 64, 3700, 256, 128), (70000, 256, 128, 128, 128), (70000, 80, 128, 128, 128), (2049, 384, 2100, 128, 128),
    (65664, 128, 64, 64, 64), (65664, 176, 64, 64, 64), (65664, 384, 61, 64, 64), (1030, 208, 1000, 64, 64),
    (333, 515, 1999, 64, 64), (333, 512, 1999, 64, 64), (70, 8192, 500, 0, 0), (1000, 208, 61, 0, 0)])
@pytest.mark.parametrize("view", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mm8_every_kernel(T, K, N, tile, side, view, dtype):
    """Every kernel with both types of result, which leave the sums by other ways: tiles of all sides whose workgroups go on
    to a next tile and to a last one, rows that end inside a step, tiles that end outside y."""
    whole = not view and K % 16 == 0
    _, names = launched(lambda: mm8_check(mm8_inputs(T, K, N, gen(T + K), view=view), dtype))
    assert names == [product(tile if whole else side, whole)]


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_through_a_gated_layer(dtype):
    """Convolution, gated recurrence and gated norm forward and back: the gradients that arrive at every input and
    parameter against the layer's in float64, which differences of its loss along themselves confirm."""
    r = gen(70)
    B, D, L, G = 2, 24, 700, 3
    x, ri, ii = (dev(r.normal(size=(B, D, L)), dtype) for _ in range(3))
    z, gy = (dev(r.normal(size=(B * L, D)), dtype) for _ in range(2))
    w, cb, nw, nb = dev(r.normal(size=(D, 4)) / 2), dev(0.1 * r.normal(size=D)), dev(1 + 0.1 * r.normal(size=D)), dev(0.1 * r.normal(size=D))
    lam = dev(np.log(np.expm1(-np.log(r.uniform(0.9, 0.999, D)))))
    rows = lambda v: v.transpose(1, 2).reshape(B * L, D).contiguous() if torch.is_tensor(v) else v.transpose(0, 2, 1).reshape(B * L, D)  # noqa: E731
    streams = lambda v: (v.reshape(B, L, D).transpose(1, 2).contiguous() if torch.is_tensor(v)  # noqa: E731
                         else v.reshape(B, L, D).transpose(0, 2, 1))
    u = ssm.conv_fwd(x=x, w=w, bias=cb, silu=True)["y"]
    h = ssm.gated_fwd(x=u, r=ri, i=ii, lam=lam, want_ckpt=True)
    norm = dict(x=rows(h["y"]), groups=G, w=nw, bias=nb, z=z, silu=True)
    gn = ssm.group_norm_bwd(gy=gy, **norm)
    gr = ssm.gated_bwd(gy=streams(gn["gx"]), x=u, r=ri, i=ii, lam=lam, ckpt=h["ckpt"])
    gc = ssm.conv_bwd(gy=gr["gx"], x=x, w=w, bias=cb, silu=True)
    got = [gc["gx"], gc["gw"], gc["gbias"], gr["gr"], gr["gi"], gr["glam"], gn["gw"], gn["gbias"], gn["gz"]]
    base = [f64(v) for v in (x, w, cb, ri, ii, lam, nw, nb, z)]

    def layer(x, w, cb, ri, ii, lam, nw, nb, z, back=False):
        u = C.conv_fwd(x, w, cb, None, True)[0]
        h = R.gated_fwd(u, ri, ii, lam, None, None, 8.0, None)["y"][0]
        n = R.norm(rows(h), G, nw, nb, 1e-5, True, z, f64(gy))
        if not back:
            return (f64(gy) * n["y"][0]).sum()
        g = R.gated_bwd(u, ri, ii, lam, None, None, 8.0, None, streams(n["gx"][0]), None)
        c = C.conv_bwd(x, w, cb, None, True, g["gx"][0], None)
        return [v[0] for v in (c["gx"], c["gw"], c["gbias"], g["gr"], g["gi"], g["glam"], n["gw"], n["gbias"], n["gz"])]

    for k, (g, v) in enumerate(zip(layer(*base, back=True), got)):
        # along itself the loss rises by |g| a unit, and an unrelated direction would not be noticed to be one; differences
        # of 1e-4 are off by 1e-8 times the loss's third derivatives, the loss itself by 1e-16 of it: 1e-12 / 1e-4
        d = g / np.linalg.norm(g)
        far = [[b + s * 1e-4 * d if j == k else b for j, b in enumerate(base)] for s in (1, -1)]
        num = (layer(*far[0]) - layer(*far[1])) / 2e-4
        assert abs(num - np.linalg.norm(g)) <= 1e-5 * np.linalg.norm(g), k
        # six roundings of streams between the stages and at the end, each at most twice as large at the gradient as where
        # it is made; fp32's own
        assert np.linalg.norm(f64(v) - g) <= (12 * R.HALF[dtype] + 1e-4) * np.linalg.norm(g), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_rows_of_any_stride(dtype):
    """Packed rows of which there are none, whatever their strides: no output rows, and the pool stays."""
    D, S = 6, 3
    none = torch.empty(0, 4 * D, dtype=DT[dtype], device=DEV)[:, ::4]
    start = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    one = dev(np.ones(D))
    for native in (False, True):   # the binding's own path (outputs come from the tests' allocator), the native calls
        if native:
            ssm.set_allocator(None)
        for f, inner, kw in (
                (ssm.tokens_conv, (D, 3), dict(x=none, w=dev(np.ones((D, 4))))),
                (ssm.tokens_scan, (D, 4), dict(delta=none, x=none, z=none, A=dev(-np.ones((D, 4))), Bm=none[:, :4], C=none[:, :4])),
                (ssm.tokens_gated, (D,), dict(x=none, r=none, i=none, lam=one))):
            pool = torch.full((S, *inner), 3.0, dtype=DT[dtype] if f is ssm.tokens_conv else torch.float32, device=DEV)
            y = f(pool=pool, seq_start=start, **kw)["y"]
            assert y.shape == (0, D) and y.dtype == DT[dtype] and (pool == 3).all()
            out = torch.empty(0, 4 * D, dtype=DT[dtype], device=DEV)[:, ::4]
            assert f(pool=pool, seq_start=start, out={"y": out}, **kw)["y"] is out and (pool == 3).all()
        assert ssm.group_norm_fwd(x=none, groups=2, z=none)["y"].shape == (0, D)
        g = ssm.group_norm_bwd(gy=none, x=none, groups=2)
        assert g["gx"].shape == (0, D) and (g["gw"] == 0).all() and (g["gbias"] == 0).all()
        assert ssm.tokens_pack8(none)["x8"].shape == (0, D)


@pytest.mark.parametrize("eps,spread", [(0.0, 2.0 ** -62), (0.0, 1.0), (1e-5, 2.0 ** -62), (1e-5, 2.0 ** 54), (0.0, 2.0 ** 54)])
@pytest.mark.parametrize("G,per", [(3, 65), (2, 2056), (1, 8192)])
def test_norm_at_the_ends_of_its_range(G, per, eps, spread):
    """Deviations whose squares' sum is just inside float32's range, and spreads whose variance is, without an eps."""
    t, gy = norm_inputs(5, G * per, "f32", gen(per))
    t["x"] = t["x"] * spread
    norm_check(t, gy, G, "f32", True, eps)

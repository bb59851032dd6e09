"""Host side of the gated recurrence, the group norm and the products in 8-bit integers: refusals of the library and of the
binding, workspaces, and the references themselves.  No GPU."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_chunked_amd as ssm
from selective_state_space_chunked_amd import binding as B

from . import _gated_ref as R
from .test_abi import FAKE, status


def code(name):
    return status("SSM_ERR_" + name)


def made(cls, base, over):
    a = cls(**{k: v for k, v in base.items() if not isinstance(v, tuple)})
    for k, v in {**{k: v for k, v in base.items() if isinstance(v, tuple)}, **over}.items():
        if isinstance(v, tuple):
            for i, s in enumerate(v):
                getattr(a, k)[i] = s
        else:
            setattr(a, k, v)
    return a


def gated_args(**over):
    return made(B.GatedArgs, dict(dtype=B.SSM_F32, power=8.0, batch=2, channels=8, length=100, x=FAKE, r=2 * FAKE, i=3 * FAKE,
                                  lam=4 * FAKE, x_stride=(800, 100), r_stride=(800, 100), i_stride=(800, 100)), over)


@pytest.mark.parametrize("over,want", [
    (dict(dtype=2), "DTYPE"), (dict(batch=-1), "SHAPE"), (dict(channels=-1), "SHAPE"), (dict(length=-1), "SHAPE"),
    (dict(batch=65536), "SHAPE"), (dict(length=1 << 31), "SHAPE"), (dict(channels=1 << 24), "SHAPE"),
    (dict(batch=32, channels=(1 << 23) + 64, length=2), "SHAPE"), (dict(power=0.0), "SHAPE"), (dict(power=-1.0), "SHAPE"), (dict(power=float("nan")), "SHAPE"),
    (dict(power=float("inf")), "SHAPE"), (dict(x=None), "NULL"), (dict(r=None), "NULL"), (dict(i=None), "NULL"),
    (dict(lam=None), "NULL"), (dict(x_stride=(800, -1)), "LAYOUT"), (dict(r_stride=(1 << 40, 100)), "LAYOUT"),
    (dict(batch=1, channels=1 << 23, i_stride=(0, (1 << 40) - 1)), "LAYOUT"),   # a span that passes 64 bits
    (dict(batch=1, channels=1 << 23, x_stride=(0, 1 << 24)), "LAYOUT"),
    (dict(i=3 * FAKE + 2), "LAYOUT"), (dict(lam=4 * FAKE + 2), "LAYOUT"), (dict(r_bias=5 * FAKE + 1), "LAYOUT"),
    (dict(h0=5 * FAKE + 2), "LAYOUT"), (dict(i_bias=7 * FAKE + 3), "LAYOUT"),
])
def test_gated_refusals(over, want):
    L = B.lib()
    a = gated_args(**over)
    o = made(B.GatedFwdOut, dict(y=9 * FAKE, y_stride=(800, 100)), {})
    assert L.ssm_gated_fwd(ctypes.byref(a), ctypes.byref(o), None) == code(want), L.ssm_last_error_detail()
    i = made(B.GatedBwdIn, dict(gy=10 * FAKE, gy_stride=(800, 100)), {})
    g = made(B.GatedGrads, dict(gx=9 * FAKE, gx_stride=(800, 100)), {})
    assert L.ssm_gated_bwd(ctypes.byref(a), ctypes.byref(i), ctypes.byref(g), 11 * FAKE, 1 << 20, None) == code(want)


def test_gated_output_refusals():
    L = B.lib()
    a = gated_args()

    def fwd(y_stride=(800, 100), **o):
        return L.ssm_gated_fwd(ctypes.byref(a), ctypes.byref(made(B.GatedFwdOut, dict(y_stride=y_stride), o)), None)

    def bwd(ws=20 * FAKE, n=1 << 20, gy=10 * FAKE, **g):
        i = made(B.GatedBwdIn, dict(gy=gy, gy_stride=(800, 100)), {k: g.pop(k) for k in ("gh_last", "ckpt") if k in g})
        s = {k: (800, 100) for k in ("gx_stride", "gr_stride", "gi_stride")}
        return L.ssm_gated_bwd(ctypes.byref(a), ctypes.byref(i), ctypes.byref(made(B.GatedGrads, s, g)), ws, n, None)

    assert L.ssm_gated_fwd(None, None, None) == code("NULL") and L.ssm_gated_fwd(ctypes.byref(a), None, None) == code("NULL")
    assert fwd() == 0 and bwd() == 0                                     # nothing wanted
    assert fwd(y=FAKE + 64) == code("LAYOUT") and fwd(y=9 * FAKE + 2) == code("LAYOUT")
    assert fwd(y=9 * FAKE, h_last=9 * FAKE + 400) == code("LAYOUT") and fwd(ckpt=4 * FAKE + 16) == code("LAYOUT")
    for bad in ((800, 0), (0, 100), (800, 99), (700, 100), (100, 100)):
        assert fwd(y=9 * FAKE, y_stride=bad) == code("LAYOUT"), bad
    assert bwd(gy=None, gx=9 * FAKE) == code("NULL") and bwd(gx=10 * FAKE) == code("LAYOUT")
    assert bwd(gh0=12 * FAKE + 2) == code("LAYOUT") and bwd(gh_last=12 * FAKE + 2, gx=9 * FAKE) == code("LAYOUT")
    assert bwd(ckpt=12 * FAKE + 1, gx=9 * FAKE) == code("LAYOUT") and bwd(gx=9 * FAKE, gr=9 * FAKE + 64) == code("LAYOUT")
    n = ctypes.c_size_t(0)
    assert L.ssm_workspace_bytes(B.SSM_OP_GATED_BWD, ctypes.byref(a), ctypes.byref(n)) == 0 and n.value >= 3 * 16 * 4 + 16 * 4
    assert bwd(ws=None, glam=12 * FAKE) == code("WORKSPACE") and bwd(n=n.value - 1, glam=12 * FAKE) == code("WORKSPACE")
    assert bwd(ws=20 * FAKE + 64, glam=12 * FAKE) == code("LAYOUT")
    assert L.ssm_workspace_bytes(B.SSM_OP_GATED_FWD, ctypes.byref(a), ctypes.byref(n)) == 0 and n.value == 0


def tgated_args(**over):
    return made(B.TokensGatedArgs, dict(dtype=B.SSM_F32, power=8.0, tokens=10, channels=8, sequences=3, slots=5, x=FAKE,
                                        r=2 * FAKE, i=3 * FAKE, lam=4 * FAKE, seq_start=5 * FAKE, slot=6 * FAKE,
                                        pool=7 * FAKE, y=8 * FAKE, x_stride=8, r_stride=8, i_stride=8, y_stride=8,
                                        pool_stride=8), over)


@pytest.mark.parametrize("over,want", [
    (dict(dtype=2), "DTYPE"), (dict(tokens=-1), "SHAPE"), (dict(slots=-1), "SHAPE"), (dict(tokens=1 << 30), "SHAPE"),
    (dict(power=0.0), "SHAPE"), (dict(seq_start=None), "SHAPE"), (dict(slot=None, slots=2), "SHAPE"),
    (dict(seq_start=None, tokens=1 << 23, sequences=1 << 23, slots=1 << 23, channels=1 << 20, pool_stride=1 << 20,
          y_stride=1 << 20), "SHAPE"),
    (dict(pool_stride=7), "LAYOUT"), (dict(y_stride=7), "LAYOUT"), (dict(x_stride=-8), "LAYOUT"),
    (dict(r_stride=1 << 40), "LAYOUT"), (dict(x=None), "NULL"), (dict(r=None), "NULL"), (dict(i=None), "NULL"),
    (dict(lam=None), "NULL"), (dict(pool=None), "NULL"), (dict(y=None), "NULL"), (dict(y=FAKE + 32), "LAYOUT"),
    (dict(pool=8 * FAKE + 32), "LAYOUT"), (dict(pool=5 * FAKE - 64), "LAYOUT"), (dict(seq_start=5 * FAKE + 2), "LAYOUT"),
    (dict(i=3 * FAKE + 2), "LAYOUT"), (dict(i_bias=9 * FAKE + 2), "LAYOUT"), (dict(pool=7 * FAKE + 2), "LAYOUT"),
])
def test_tokens_gated_refusals(over, want):
    L = B.lib()
    a = tgated_args(**over)
    assert L.ssm_tokens_gated(ctypes.byref(a), 20 * FAKE, 1 << 30, None) == code(want), L.ssm_last_error_detail()


def test_tokens_gated_workspace_and_empty():
    L = B.lib()
    assert L.ssm_tokens_gated(None, None, 0, None) == code("NULL")
    n = ctypes.c_size_t(0)
    a = tgated_args()
    assert L.ssm_workspace_bytes(B.SSM_OP_TOKENS_GATED, ctypes.byref(a), ctypes.byref(n)) == 0 and n.value > 0
    assert L.ssm_tokens_gated(ctypes.byref(a), None, 0, None) == code("WORKSPACE")
    assert L.ssm_tokens_gated(ctypes.byref(a), 20 * FAKE, n.value - 1, None) == code("WORKSPACE")
    assert L.ssm_tokens_gated(ctypes.byref(a), 20 * FAKE + 16, n.value, None) == code("LAYOUT")
    step = tgated_args(seq_start=None, tokens=3)
    assert L.ssm_workspace_bytes(B.SSM_OP_TOKENS_GATED, ctypes.byref(step), ctypes.byref(n)) == 0 and n.value == 0
    for over in (dict(tokens=0), dict(channels=0, pool_stride=0), dict(sequences=0), dict(slots=0)):   # nothing is touched
        assert L.ssm_tokens_gated(ctypes.byref(tgated_args(x=None, y=None, **over)), None, 0, None) == 0


def norm_args(**over):
    return made(B.GroupNormArgs, dict(dtype=B.SSM_F32, rows=10, channels=24, groups=3, x=FAKE, z=2 * FAKE, w=3 * FAKE,
                                      bias=4 * FAKE, x_stride=24, z_stride=24, eps=1e-5), over)


@pytest.mark.parametrize("over,want", [
    (dict(dtype=7), "DTYPE"), (dict(rows=-1), "SHAPE"), (dict(groups=0), "SHAPE"), (dict(groups=5), "SHAPE"),
    (dict(rows=1 << 30), "SHAPE"), (dict(channels=1 << 24, groups=1 << 20), "SHAPE"), (dict(silu=2), "SHAPE"),
    (dict(eps=-1.0), "SHAPE"), (dict(eps=float("nan")), "SHAPE"), (dict(channels=8193, groups=1, x_stride=8193, z_stride=8193), "UNSUPPORTED"),
    (dict(x=None), "NULL"), (dict(x_stride=-1), "LAYOUT"), (dict(z_stride=1 << 40), "LAYOUT"), (dict(x=FAKE + 2), "LAYOUT"),
    (dict(z=2 * FAKE + 1), "LAYOUT"), (dict(w=3 * FAKE + 2), "LAYOUT"), (dict(bias=4 * FAKE + 2), "LAYOUT"),
])
def test_norm_refusals(over, want):
    L = B.lib()
    a = norm_args(**over)
    width = 24 if a.channels < 8000 else a.channels
    assert L.ssm_group_norm_fwd(ctypes.byref(a), 6 * FAKE, width, None) == code(want), L.ssm_last_error_detail()
    g = B.GroupNormGrads(gx=7 * FAKE, gx_stride=width)
    assert L.ssm_group_norm_bwd(ctypes.byref(a), 8 * FAKE, width, ctypes.byref(g), 9 * FAKE, 1 << 24, None) == code(want)


def test_norm_output_refusals():
    L = B.lib()
    a = norm_args()

    def bwd(gy=8 * FAKE, ws=9 * FAKE, n=1 << 20, a=a, **g):
        return L.ssm_group_norm_bwd(ctypes.byref(a), gy, 24, ctypes.byref(B.GroupNormGrads(gx_stride=24, gz_stride=24, **g)),
                                    ws, n, None) if "gx_stride" not in g else \
            L.ssm_group_norm_bwd(ctypes.byref(a), gy, 24, ctypes.byref(B.GroupNormGrads(gz_stride=24, **g)), ws, n, None)

    assert L.ssm_group_norm_fwd(None, 6 * FAKE, 24, None) == code("NULL")
    assert L.ssm_group_norm_fwd(ctypes.byref(a), None, 24, None) == code("NULL")
    assert L.ssm_group_norm_fwd(ctypes.byref(a), 6 * FAKE, 23, None) == code("LAYOUT")
    assert L.ssm_group_norm_fwd(ctypes.byref(a), FAKE + 64, 24, None) == code("LAYOUT")
    assert bwd() == 0                                                    # nothing wanted
    assert bwd(gy=None, gx=7 * FAKE) == code("NULL") and bwd(gx=8 * FAKE) == code("LAYOUT")
    assert bwd(gx=7 * FAKE, gx_stride=20) == code("LAYOUT") and bwd(gz=7 * FAKE, a=norm_args(z=None)) == code("NULL")
    assert bwd(gw=7 * FAKE + 2) == code("LAYOUT") and bwd(gw=7 * FAKE, gbias=7 * FAKE + 4) == code("LAYOUT")
    n = ctypes.c_size_t(0)
    assert L.ssm_workspace_bytes(B.SSM_OP_GROUP_NORM_BWD, ctypes.byref(a), ctypes.byref(n)) == 0 and n.value >= 2 * 24 * 4
    assert bwd(gw=7 * FAKE, n=n.value - 1) == code("WORKSPACE") and bwd(gw=7 * FAKE, ws=None) == code("WORKSPACE")


def pack8_args(**over):
    return made(B.TokensPack8Args, dict(dtype=B.SSM_F32, tokens=4, channels=20, x=FAKE, x8=2 * FAKE, x8_scale=3 * FAKE,
                                        x_stride=20, x8_stride=20), over)


def mm8_args(**over):
    return made(B.TokensMm8Args, dict(dtype=B.SSM_F32, tokens=4, inputs=20, outputs=6, x8=FAKE, x8_scale=2 * FAKE,
                                      w8=3 * FAKE, w8_scale=4 * FAKE, y=5 * FAKE, x8_stride=20, w8_stride=20, y_stride=6), over)


def test_mm8_refusals():
    L = B.lib()
    for over, want in ((dict(dtype=3), "DTYPE"), (dict(tokens=-1), "SHAPE"), (dict(channels=1 << 17, x_stride=1 << 17, x8_stride=1 << 17), "SHAPE"),
                       (dict(tokens=1 << 24), "SHAPE"), (dict(x=None), "NULL"), (dict(x8=None), "NULL"),
                       (dict(x8_scale=None), "NULL"), (dict(x8_stride=19), "LAYOUT"), (dict(x_stride=-1), "LAYOUT"),
                       (dict(x=FAKE + 2), "LAYOUT"), (dict(x8=FAKE + 8), "LAYOUT"), (dict(x8_scale=2 * FAKE + 4), "LAYOUT"),
                       (dict(x8_scale=3 * FAKE + 2), "LAYOUT")):
        assert L.ssm_tokens_pack8(ctypes.byref(pack8_args(**over)), None) == code(want), over
    for over, want in ((dict(dtype=3), "DTYPE"), (dict(outputs=-1), "SHAPE"), (dict(inputs=1 << 17, x8_stride=1 << 17, w8_stride=1 << 17), "SHAPE"),
                       (dict(outputs=1 << 26, y_stride=1 << 26), "SHAPE"), (dict(tokens=1 << 20, outputs=1 << 17, y_stride=1 << 17), "SHAPE"),
                       (dict(x8=None), "NULL"), (dict(w8=None), "NULL"), (dict(x8_scale=None), "NULL"),
                       (dict(w8_scale=None), "NULL"), (dict(y=None), "NULL"), (dict(y_stride=5), "LAYOUT"),
                       (dict(w8_stride=-1), "LAYOUT"), (dict(y=FAKE + 32), "LAYOUT"), (dict(y=5 * FAKE + 2), "LAYOUT"),
                       (dict(w8_scale=4 * FAKE + 1), "LAYOUT"), (dict(bias=7 * FAKE + 2), "LAYOUT"),
                       (dict(bias=5 * FAKE + 16), "LAYOUT")):
        assert L.ssm_tokens_mm8(ctypes.byref(mm8_args(**over)), None) == code(want), over
    assert L.ssm_tokens_pack8(None, None) == code("NULL") and L.ssm_tokens_mm8(None, None) == code("NULL")
    assert L.ssm_tokens_pack8(ctypes.byref(pack8_args(tokens=0, x=None, x8=None, x8_scale=None)), None) == 0
    for over in (dict(tokens=0), dict(outputs=0, y_stride=0)):
        assert L.ssm_tokens_mm8(ctypes.byref(mm8_args(x8=None, w8=None, y=None, **over)), None) == 0


@pytest.mark.parametrize("packed,cls", [
    (B._GATED_ARGS, B.GatedArgs), (B._GATED_IO, B.GatedFwdOut), (B._GATED_IO, B.GatedBwdIn), (B._GATED_GRADS, B.GatedGrads),
    (B._TOKENS_GATED_ARGS, B.TokensGatedArgs), (B._GROUP_NORM_ARGS, B.GroupNormArgs), (B._GROUP_NORM_GRADS, B.GroupNormGrads),
    (B._TOKENS_PACK8_ARGS, B.TokensPack8Args), (B._TOKENS_MM8_ARGS, B.TokensMm8Args)])
def test_packed_arguments_are_the_structs(packed, cls):
    """Every field at its place."""
    fields = []
    for name, t in cls._fields_:
        fields += [(name, i) for i in range(2)] if t is ctypes.c_int64 * 2 else [(name, None)]
    got = cls.from_buffer_copy(packed.pack(*range(1, len(fields) + 1)))
    assert ctypes.sizeof(cls) == packed.size
    for k, (name, i) in enumerate(fields):
        v = getattr(got, name)
        assert (v if i is None else v[i]) == k + 1, name


def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses():
    x = t(2, 3, 9)
    g = dict(x=x, r=x.clone(), i=x.clone(), lam=t(3))
    for over, err in ((dict(), ValueError),                                       # host tensors
                      (dict(x=t(2, 3)), ValueError), (dict(x=x.half()), TypeError), (dict(x=None), ValueError),
                      (dict(r=t(2, 3, 8)), ValueError), (dict(r=x.bfloat16()), TypeError), (dict(i=None), ValueError),
                      (dict(i=t(2, 3, 18)[..., ::2]), ValueError), (dict(lam=None), ValueError), (dict(lam=t(4)), ValueError),
                      (dict(lam=t(3).double()), TypeError), (dict(r_bias=t(2)), ValueError), (dict(h0=t(2, 4)), ValueError),
                      (dict(power="x"), ValueError)):
        with pytest.raises(err):
            ssm.gated_fwd(**{**g, **over})
        with pytest.raises(err):
            ssm.gated_bwd(gy=t(2, 3, 9), **{**g, **over})
    with pytest.raises(ValueError, match="unknown gradient"):
        ssm.gated_bwd(gy=t(2, 3, 9), want=("gq",), **g)
    with pytest.raises(TypeError):
        ssm.gated_bwd(gy=t(2, 3, 9).bfloat16(), **g)
    with pytest.raises(ValueError):
        ssm.gated_bwd(gy=t(2, 3, 9), ckpt=t(2, 3, 2), **g)
    with pytest.raises(ValueError, match="distinct"):
        ssm.gated_fwd(out={"y": t(1, 3, 9).expand(2, 3, 9)}, **g)

    rows = dict(x=t(5, 8), r=t(5, 8), i=t(5, 8), lam=t(8), pool=t(6, 8))
    for over, err in ((dict(), ValueError), (dict(x=t(5, 8, 1)), ValueError), (dict(pool=t(6, 8, 1)), ValueError),
                      (dict(pool=t(6, 7)), ValueError), (dict(pool=t(6, 8).bfloat16()), TypeError),
                      (dict(pool=t(6, 16)[:, ::2]), ValueError), (dict(slot=t(5)), TypeError),
                      (dict(seq_start=t(3)), TypeError), (dict(fresh=t(5)), TypeError), (dict(r=t(4, 8)), ValueError),
                      (dict(lam=None), ValueError), (dict(out={"y": t(5, 7)}), ValueError)):
        with pytest.raises(err):
            ssm.tokens_gated(**{**rows, **over})

    n = dict(x=t(5, 12), groups=3)
    for over, err in ((dict(), ValueError), (dict(x=t(5)), ValueError), (dict(groups=2.0), TypeError), (dict(w=t(11)), ValueError),
                      (dict(bias=t(12).double()), TypeError), (dict(z=t(5, 11)), ValueError), (dict(z=t(5, 12).bfloat16()), TypeError),
                      (dict(x=t(5, 12).half()), TypeError)):
        with pytest.raises(err):
            ssm.group_norm_fwd(**{**n, **over})
        with pytest.raises(err):
            ssm.group_norm_bwd(gy=t(5, 12), **{**n, **over})
    with pytest.raises(ValueError, match="unknown gradient"):
        ssm.group_norm_bwd(gy=t(5, 12), want=("gy",), **n)

    i8 = torch.int8
    m = dict(x8=t(4, 6, dtype=i8), x8_scale=t(4), w8=t(3, 6, dtype=i8), w8_scale=t(3))
    for over, err in ((dict(), ValueError), (dict(x8=t(4, 6)), TypeError), (dict(w8=t(3, 5, dtype=i8)), ValueError),
                      (dict(x8=t(4, dtype=i8)), ValueError), (dict(w8=None), ValueError), (dict(x8_scale=None), ValueError),
                      (dict(w8_scale=t(4)), ValueError), (dict(bias=t(4)), ValueError), (dict(dtype=torch.float16), TypeError),
                      (dict(out={"y": t(4, 3)}), TypeError)):
        with pytest.raises(err):
            ssm.tokens_mm8(**{**m, **over})
    for x in (t(4), t(4, 6).half(), t(4, 6), None):
        with pytest.raises((ValueError, TypeError)):
            ssm.tokens_pack8(x)


def test_reference_gradients_by_differences():
    """The references' gradients against central differences of their forwards."""
    r = np.random.default_rng(0)
    v = dict(x=r.normal(size=(2, 3, 20)), r=r.normal(size=(2, 3, 20)), i=r.normal(size=(2, 3, 20)), lam=r.normal(size=3) - 3,
             r_bias=r.normal(size=3), i_bias=r.normal(size=3))
    h0, gy, gl = r.normal(size=(2, 3)), r.normal(size=(2, 3, 20)), r.normal(size=(2, 3))

    def loss(v, h0):
        f = R.gated_fwd(*v.values(), 8.0, h0)
        return (gy * f["y"][0]).sum() + (gl * f["h_last"][0]).sum()

    g = R.gated_bwd(*v.values(), 8.0, h0, gy, gl)
    for k, n in {"gx": "x", "gr": "r", "gi": "i", "glam": "lam", "gr_bias": "r_bias", "gi_bias": "i_bias"}.items():
        d = r.normal(size=v[n].shape)
        num = (loss({**v, n: v[n] + 1e-6 * d}, h0) - loss({**v, n: v[n] - 1e-6 * d}, h0)) / 2e-6
        assert abs(num - (g[k][0] * d).sum()) <= 1e-6 * max(1, abs(num)), k
    d = r.normal(size=h0.shape)
    num = (loss(v, h0 + 1e-6 * d) - loss(v, h0 - 1e-6 * d)) / 2e-6
    assert abs(num - (g["gh0"][0] * d).sum()) <= 1e-6 * max(1, abs(num))

    n = dict(x=r.normal(size=(4, 12)), w=r.normal(size=12), bias=r.normal(size=12), z=r.normal(size=(4, 12)))
    gy = r.normal(size=(4, 12))
    for act in (False, True):
        def nloss(n):
            return (gy * R.norm(n["x"], 3, n["w"], n["bias"], 1e-5, act, n["z"])["y"][0]).sum()
        g = R.norm(n["x"], 3, n["w"], n["bias"], 1e-5, act, n["z"], gy)
        for k, m in {"gx": "x", "gw": "w", "gbias": "bias", "gz": "z"}.items():
            d = r.normal(size=n[m].shape)
            num = (nloss({**n, m: n[m] + 1e-6 * d}) - nloss({**n, m: n[m] - 1e-6 * d})) / 2e-6
            assert abs(num - (g[k][0] * d).sum()) <= 1e-6 * max(1, abs(num)), k

"""The short convolution, 8-bit checkpoints and packed-row forms without a GPU: their refusals, before anything is
enqueued, and the float64 references against differences and against the fp64 scan oracle."""
import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import selective_state_space_chunked_amd as ssm
from selective_state_space_chunked_amd import binding as B

from . import _layer_ref as R

FAKE = 1 << 30   # never dereferenced


def code(name):
    return {"NULL": -1, "SHAPE": -2, "DTYPE": -3, "LAYOUT": -4, "WORKSPACE": -5, "UNSUPPORTED": -6}[name]


def conv_args(**over):
    a = B.ConvArgs(dtype=B.SSM_F32, silu=1, batch=2, channels=8, length=100, width=4, x=FAKE, w=2 * FAKE, bias=3 * FAKE)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def lay(**roles):
    v = B.Layout()
    for k, st in roles.items():
        r = getattr(B, "V_" + k)
        v.given |= 1 << r
        for i, s in enumerate(st):
            v.stride[r][i] = s
    return ctypes.pointer(v)


@pytest.mark.parametrize("over,want", [
    (dict(dtype=2), "DTYPE"), (dict(width=1), "UNSUPPORTED"), (dict(width=5), "UNSUPPORTED"),
    (dict(batch=-1), "SHAPE"), (dict(batch=65536), "SHAPE"), (dict(length=1 << 31), "SHAPE"), (dict(silu=2), "SHAPE"),
    (dict(batch=8, length=1 << 30), "SHAPE"),
    (dict(x=None), "NULL"), (dict(w=None), "NULL"), (dict(x8=4 * FAKE), "SHAPE"), (dict(x=None, x8=4 * FAKE), "NULL"),
    (dict(x=FAKE + 2), "LAYOUT"), (dict(w=FAKE * 2 + 2), "LAYOUT"), (dict(init=FAKE * 5 + 1), "LAYOUT"),
    (dict(layout=lay(X=(800, 100, 2))), "LAYOUT"), (dict(layout=lay(X=(800, -100, 1))), "LAYOUT"),
    (dict(layout=lay(BM=(1, 1, 1, 1))), "UNSUPPORTED"), (dict(layout=lay(GX=(800, 100, 1))), "UNSUPPORTED"),
    (dict(x=None, x8=4 * FAKE, x8_scale=5 * FAKE, layout=lay(X=(801, 100, 1))), "UNSUPPORTED"),
])
def test_conv_refusals(over, want):
    a = conv_args(**over)
    o = B.ConvFwdOut(y=6 * FAKE)
    assert B.lib().ssm_conv_fwd(ctypes.byref(a), ctypes.byref(o), None) == code(want), B.lib().ssm_last_error_detail()
    assert B.lib().ssm_last_error_detail()


def test_conv_output_refusals():
    L = B.lib()
    a = conv_args()

    def fwd(**o):
        return L.ssm_conv_fwd(ctypes.byref(a), ctypes.byref(B.ConvFwdOut(**o)), None)

    def bwd(gy=7 * FAKE, glast=None, ws=None, n=0, **g):
        return L.ssm_conv_bwd(ctypes.byref(a), gy, glast, ctypes.byref(B.ConvGrads(**g)), ws, n, None)

    assert L.ssm_conv_fwd(ctypes.byref(a), None, None) == code("NULL")
    assert L.ssm_conv_fwd(None, None, None) == code("NULL")
    assert fwd(x8=6 * FAKE) == code("NULL") and fwd(x8_scale=6 * FAKE) == code("NULL")
    assert fwd(y=FAKE + 64) == code("LAYOUT")                       # over x
    assert fwd(y=6 * FAKE, last=6 * FAKE + 4) == code("LAYOUT")     # over another output
    assert fwd(y=6 * FAKE + 2) == code("LAYOUT")
    assert fwd() == 0                                               # nothing wanted
    assert bwd(gy=None, gx=6 * FAKE) == code("NULL")
    assert bwd(gx=7 * FAKE) == code("LAYOUT")
    assert bwd(gw=6 * FAKE + 2) == code("LAYOUT")
    n = ctypes.c_size_t(0)
    assert L.ssm_workspace_bytes(B.SSM_OP_CONV_BWD, ctypes.byref(a), ctypes.byref(n)) == 0
    big = conv_args(batch=8, channels=2, length=100000)             # few channels: sums in parts
    assert L.ssm_workspace_bytes(B.SSM_OP_CONV_BWD, ctypes.byref(big), ctypes.byref(n)) == 0 and n.value > 0
    g = B.ConvGrads(gw=9 * FAKE)
    assert L.ssm_conv_bwd(ctypes.byref(big), 7 * FAKE, None, ctypes.byref(g), None, 0, None) == code("WORKSPACE")
    assert L.ssm_conv_bwd(ctypes.byref(big), 7 * FAKE, None, ctypes.byref(g), 8 * FAKE, n.value - 1, None) == code("WORKSPACE")
    assert L.ssm_conv_bwd(ctypes.byref(big), 7 * FAKE, None, ctypes.byref(g), 8 * FAKE + 64, n.value, None) == code("LAYOUT")
    assert L.ssm_workspace_bytes(B.SSM_OP_CONV_FWD, ctypes.byref(a), ctypes.byref(n)) == 0 and n.value == 0


def test_ckpt8_refusals():
    L = B.lib()
    a = B.Ckpt8Args(dtype=B.SSM_F32, batch=2, channels=8, length=100)
    assert L.ssm_ckpt8_pack(None, FAKE, 2 * FAKE, 3 * FAKE, None) == code("NULL")
    assert L.ssm_ckpt8_pack(ctypes.byref(a), FAKE, None, 3 * FAKE, None) == code("NULL")
    assert L.ssm_ckpt8_pack(ctypes.byref(a), FAKE, FAKE + 64, 3 * FAKE, None) == code("LAYOUT")
    assert L.ssm_ckpt8_unpack(ctypes.byref(a), FAKE, 2 * FAKE + 1, 3 * FAKE, None) == code("LAYOUT")
    assert L.ssm_ckpt8_unpack(ctypes.byref(a), FAKE, 2 * FAKE, FAKE - 64, None) == code("LAYOUT")
    a.dtype = 5
    assert L.ssm_ckpt8_unpack(ctypes.byref(a), FAKE, 2 * FAKE, 3 * FAKE, None) == code("DTYPE")


def tconv_args(**over):
    a = B.TokensConvArgs(dtype=B.SSM_F32, silu=1, tokens=10, channels=8, width=4, sequences=3, slots=5, x=FAKE,
                         w=2 * FAKE, seq_start=3 * FAKE, slot=4 * FAKE, pool=5 * FAKE, y=6 * FAKE, x_stride=8,
                         y_stride=8, pool_stride=24)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def tscan_args(**over):
    a = B.TokensScanArgs(dtype=B.SSM_F32, tokens=10, channels=8, state=16, sequences=3, slots=5, delta=7 * FAKE, x=FAKE,
                         A=2 * FAKE, Bm=8 * FAKE, C=9 * FAKE, seq_start=3 * FAKE, slot=4 * FAKE, pool=5 * FAKE,
                         y=6 * FAKE, delta_stride=8, x_stride=8, Bm_stride=16, C_stride=16, y_stride=8, pool_stride=128)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,want", [
    (dict(dtype=2), "DTYPE"), (dict(tokens=-1), "SHAPE"), (dict(slots=-1), "SHAPE"), (dict(tokens=1 << 30), "SHAPE"),
    (dict(seq_start=None), "SHAPE"),                          # 10 rows, 3 sequences
    (dict(slot=None, slots=2), "SHAPE"),                      # fewer slots than sequences
    (dict(pool_stride=23), "LAYOUT"), (dict(y_stride=7), "LAYOUT"), (dict(x_stride=-8), "LAYOUT"),
    (dict(x=None), "NULL"), (dict(pool=None), "NULL"), (dict(y=None), "NULL"),
    (dict(y=FAKE + 32), "LAYOUT"), (dict(pool=FAKE + 32), "LAYOUT"), (dict(pool=6 * FAKE + 32), "LAYOUT"),
    (dict(pool=3 * FAKE - 64), "LAYOUT"), (dict(seq_start=3 * FAKE + 2), "LAYOUT"), (dict(x=FAKE + 2), "LAYOUT"),
])
def test_tokens_refusals(over, want):
    L = B.lib()
    a = tconv_args(**over)
    assert L.ssm_tokens_conv(ctypes.byref(a), None) == code(want), L.ssm_last_error_detail()
    over = dict(over)
    if over.get("pool_stride"):
        over["pool_stride"] = 127
    a = tscan_args(**over)
    assert L.ssm_tokens_scan(ctypes.byref(a), None, 0, None) == code(want), L.ssm_last_error_detail()


def test_tokens_own_refusals():
    L = B.lib()
    assert L.ssm_tokens_conv(None, None) == code("NULL") and L.ssm_tokens_scan(None, None, 0, None) == code("NULL")
    for width in (1, 5):
        assert L.ssm_tokens_conv(ctypes.byref(tconv_args(width=width)), None) == code("UNSUPPORTED")
    for over, want in ((dict(state=0), "SHAPE"), (dict(state=17), "SHAPE"), (dict(delta_softplus=3), "SHAPE"),
                       (dict(delta=None), "NULL"), (dict(Bm=None), "NULL"), (dict(z=FAKE + 2, z_stride=8), "LAYOUT"),
                       (dict(C_stride=-1), "LAYOUT"), (dict(skip=5 * FAKE + 64), "LAYOUT"),
                       (dict(A=2 * FAKE + 1), "LAYOUT")):
        assert L.ssm_tokens_scan(ctypes.byref(tscan_args(**over)), None, 0, None) == code(want), over
    for over in (dict(tokens=0), dict(channels=0, pool_stride=0), dict(sequences=0), dict(slots=0)):   # empty: nothing is touched
        assert L.ssm_tokens_conv(ctypes.byref(tconv_args(x=None, y=None, **over)), None) == 0
        assert L.ssm_tokens_scan(ctypes.byref(tscan_args(x=None, y=None, **over)), None, 0, None) == 0


def _t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses():
    """The binding's own checks, before the library is called."""
    x, w = _t(2, 3, 10), _t(3, 4)
    with pytest.raises(ValueError, match="GPU"):
        ssm.conv_fwd(x=x, w=w)
    with pytest.raises(ValueError, match="GPU"):
        ssm.ckpt8_pack(x)
    for kw, exc in ((dict(x=x, w=_t(2, 4)), ValueError), (dict(w=w), ValueError),
                    (dict(x=x, w=w, init=_t(2, 3, 4)), ValueError), (dict(x=x.double(), w=w), TypeError),
                    (dict(x=x, w=w, bias=_t(4)), ValueError), (dict(x=x.transpose(1, 2), w=_t(10, 4)), ValueError),
                    (dict(ckpt8=(_t(2, 3, 10, dtype=torch.int8), _t(2, 3, 2)), w=w, dtype=torch.float32), ValueError),
                    (dict(ckpt8=(_t(2, 3, 10, dtype=torch.int8), _t(2, 3, 1)), w=w), TypeError),
                    (dict(x=x, ckpt8=(_t(2, 3, 10, dtype=torch.int8), _t(2, 3, 1)), w=w), ValueError),
                    (dict(ckpt8=(_t(2, 3, 10, dtype=torch.int8), _t(2, 3, 1)), w=w, dtype=torch.float32,
                          want_ckpt8=True), ValueError),
                    (dict(x=x, w=w, out={"y": x[:1].expand(2, 3, 10)}), ValueError)):
        with pytest.raises(exc):
            ssm.conv_fwd(**kw)
    with pytest.raises(ValueError):
        ssm.conv_bwd(gy=x, x=x, w=w, want=("gz",))
    with pytest.raises(TypeError):
        ssm.conv_bwd(gy=x.bfloat16(), x=x, w=w)
    r = _t(6, 3)
    pool = _t(4, 3, 3)
    i32 = dict(dtype=torch.int32)
    good = dict(x=r, w=w, pool=pool, seq_start=_t(3, **i32), slot=_t(2, **i32))
    for over, exc in ((dict(pool=_t(4, 3, 2)), ValueError), (dict(pool=pool.bfloat16()), TypeError),
                      (dict(seq_start=_t(3)), TypeError), (dict(slot=_t(3, **i32)), ValueError),
                      (dict(fresh=_t(2)), TypeError), (dict(fresh=[True, False]), ValueError),
                      (dict(x=_t(2, 6, 3)), ValueError),
                      (dict(pool=_t(4, 3, 6)[..., ::2]), ValueError), (dict(seq_start=_t(0, **i32)), ValueError),
                      (dict(), ValueError)):       # the last: host tensors
        with pytest.raises(exc):
            ssm.tokens_conv(**{**good, **over})
    p2 = _t(4, 3, 5)
    good = dict(delta=r, x=r, A=_t(3, 5), Bm=_t(6, 5), C=_t(6, 5), pool=p2, seq_start=_t(3, **i32), slot=_t(2, **i32))
    for over, exc in ((dict(Bm=_t(6, 4)), ValueError), (dict(delta=r.bfloat16()), TypeError), (dict(C=None), ValueError),
                      (dict(pool=p2.bfloat16()), TypeError), (dict(z=_t(5, 3)), ValueError),
                      (dict(A=_t(4, 5)), ValueError), (dict(skip=_t(5)), ValueError), (dict(), ValueError)):
        with pytest.raises(exc):
            ssm.tokens_scan(**{**good, **over})


# ---------------------------------------------------------------------------
# the references
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("L,W", [(1, 4), (2, 4), (3, 2), (17, 3)])
def test_reference_gradients_by_differences(L, W, silu):
    rng = np.random.default_rng(L * 10 + W)
    v = {"x": rng.normal(size=(2, 3, L)), "w": rng.normal(size=(3, W)), "bias": rng.normal(size=3),
         "init": rng.normal(size=(2, 3, W - 1))}
    gy, gl = rng.normal(size=(2, 3, L)), rng.normal(size=(2, 3, W - 1))

    def loss(**over):
        a = {**v, **over}
        y, _, last = R.conv_fwd(a["x"], a["w"], a["bias"], a["init"], silu)
        return (y * gy).sum() + (last * gl).sum()

    g = R.conv_bwd(v["x"], v["w"], v["bias"], v["init"], silu, gy, gl)
    for k, name in (("x", "gx"), ("w", "gw"), ("bias", "gbias"), ("init", "ginit")):
        for i in np.ndindex(v[k].shape):
            d = np.zeros_like(v[k])
            d[i] = 1e-5
            # central difference: h^2 / 6 times the third derivative (a few), and 1e-16 / h of rounding
            assert abs((loss(**{k: v[k] + d}) - loss(**{k: v[k] - d})) / 2e-5 - g[name][0][i]) < 1e-7, (name, i)


def test_reference_scan_is_the_oracles():
    """One sequence without gate and skip, against the fp64 oracle of the library's selective scan."""
    rng = np.random.default_rng(5)
    T, D, N = 23, 4, 5
    delta, x = rng.uniform(0.01, 0.5, (T, D)), rng.normal(size=(T, D))
    A, Bm, C, h0 = -rng.uniform(0.5, 4, (D, N)), rng.normal(size=(T, N)), rng.normal(size=(T, N)), rng.normal(size=(1, D, N))
    f32 = lambda a: np.ascontiguousarray(a, np.float32)  # noqa: E731
    y0, h0_last = oracle.real_fwd(delta=f32(delta.T[None]), x=f32(x.T[None]), A=f32(A), Bm=f32(Bm[None]), C=f32(C[None]),
                                  h0=f32(h0), B=1, D=D, L=T, N=N)
    v = [f32(a).astype(np.float64) for a in (delta, x, A, Bm, C)]
    y, _, pool, _ = R.tokens_scan(*v, None, None, None, False, f32(h0).astype(np.float64), [0, T], [0], None,
                                  np.zeros((T, D)))
    np.testing.assert_allclose(y.T[None], y0, rtol=1e-12, atol=1e-13)   # both in fp64
    np.testing.assert_allclose(pool, h0_last, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("packed,struct", [("_CONV_ARGS", "ConvArgs"), ("_FOUR_PTRS", "ConvFwdOut"),
                                           ("_FOUR_PTRS", "ConvGrads"), ("_CKPT8_ARGS", "Ckpt8Args"),
                                           ("_TOKENS_CONV_ARGS", "TokensConvArgs"),
                                           ("_TOKENS_SCAN_ARGS", "TokensScanArgs")])
def test_packed_arguments_are_the_structs(packed, struct):
    """The bytes the binding passes are the struct's, field by field."""
    p, c = getattr(B, packed), getattr(B, struct)
    assert p.size == ctypes.sizeof(c)
    n = len(p.unpack(bytes(p.size)))
    fields = [f[0] for f in c._fields_]
    assert n == len(fields)
    got = c.from_buffer_copy(p.pack(*range(1, n + 1)))
    for i, f in enumerate(fields):
        v = getattr(got, f)
        if f == "layout":
            v = ctypes.cast(v, ctypes.c_void_p).value
        assert v == i + 1, f


def test_checkpoint_error_bound():
    """Blocks whose element lies next to a half of a step: the rounding to a byte is off by 1/2, and the reciprocal step,
    the product, the scale and the value by 2^-24 of up to 127 scales each, 127 * 2^-22 < 2^-15 in all."""
    rng = np.random.default_rng(0)
    amax = np.append(rng.uniform(1, 2, 200000), 1.0524639).astype(np.float32)
    x = ((rng.integers(100, 127, amax.size) + 0.5) * amax.astype(np.float64) / 127).astype(np.float32)
    x = x.view(np.int32) + rng.integers(-4, 5, amax.size, dtype=np.int32)
    x = x.view(np.float32)
    x[-1] = 1.0317461      # off by (1/2 + 1.24 * 2^-16) scale
    block = np.stack([amax, x], -1)[None]
    q, s = R.pack(block)
    off = np.abs(R.unpack(q, s).astype(np.float64) - block) / s.astype(np.float64)
    assert off.max() <= 0.5 + 2.0 ** -15
    assert off[0, -1, 1] > 0.5 + 2.0 ** -16


@pytest.mark.parametrize("module", [None, b"no shared object"])
def test_library_without_the_native_calls(module, tmp_path):
    """The package with the HIP library alone, the native module missing or built for another interpreter: every entry
    point is there, and what wants the module warns once and goes on without it."""
    pkg = tmp_path / "selective_state_space_chunked_amd"
    pkg.mkdir()
    here = os.path.dirname(B.__file__)
    for f in os.listdir(here):
        if f.endswith(".py"):
            shutil.copy(os.path.join(here, f), pkg)
    os.symlink(B.LIB_PATH, pkg / "libssmscan.so")
    if module is not None:
        (pkg / "_pycall.so").write_bytes(module)
    code = """
import warnings
import torch
import selective_state_space_chunked_amd as ssm
from selective_state_space_chunked_amd import binding as B

with warnings.catch_warnings():
    warnings.simplefilter("error")
    assert ssm.lib().ssm_abi_version() == 8          # what the scans need
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")

    class OnGpu(torch.Tensor):
        is_cuda = True

    x = torch.zeros(1, 2, 3).as_subclass(OnGpu)
    assert B._native(x) is None and B._native(x) is None
    assert [i.category for i in w] == [RuntimeWarning] and "native calls" in str(w[0].message)
    try:
        ssm.conv_fwd(x=torch.zeros(1, 2, 3), w=torch.zeros(2, 4))
    except ValueError as e:
        assert "GPU" in str(e)
    else:
        raise AssertionError
print("went on")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0 and r.stdout == "went on\n", r.stderr


@pytest.mark.parametrize("lacks", ["torch", "compiler"])
def test_library_builds_without_the_native_calls(lacks, tmp_path, monkeypatch, capsys):
    """What only the native calls need -- torch, a host compiler with the Python headers -- the library is built without;
    native calls of an earlier build do not stay beside it."""
    from selective_state_space_chunked_amd import build

    def run(cmd, **_):
        good = not any("pycall" in c for c in cmd)
        if good:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0 if good else 1, "", "" if good else "no Python.h")

    out, native = tmp_path / "libssmscan.so", tmp_path / "_pycall.so"
    native.write_bytes(b"earlier")
    for name, value in (("OUT", str(out)), ("PYCALL", str(native)), ("BUILD_DIR", str(tmp_path / "b"))):
        monkeypatch.setattr(build, name, value)
    monkeypatch.setattr(build.subprocess, "run", run)
    if lacks == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == str(out)
    assert out.exists() and not native.exists()
    assert "without the native calls" in capsys.readouterr().err


def test_row_strides():
    """A single row's stride is not used; the step forms and the convolution take any stride below 2^40, the scan of
    prompts any below 2^26."""
    L, n = B.lib(), ctypes.c_size_t(0)

    def conv(**over):
        return L.ssm_workspace_bytes(B.SSM_OP_TOKENS_CONV, ctypes.byref(tconv_args(**over)), ctypes.byref(n))

    def scan(**over):
        return L.ssm_workspace_bytes(B.SSM_OP_TOKENS_SCAN, ctypes.byref(tscan_args(**over)), ctypes.byref(n))

    step = dict(seq_start=None, sequences=10, slots=10)
    one = dict(tokens=1, sequences=1)
    for name in ("x_stride", "y_stride", "delta_stride", "Bm_stride", "C_stride", "z_stride"):
        calls = [scan] if name not in ("x_stride", "y_stride") else [conv, scan]
        z = dict(z=10 * FAKE, z_stride=8) if name == "z_stride" else {}
        for call in calls:
            def stride(v, **over):
                return call(**{**(z if call is scan else {}), **over, name: v})

            assert stride(1 << 50, **one) == 0 and stride(0, **one) == 0 and stride(1 << 50, **one, seq_start=None) == 0
            assert stride(1 << 26, **step) == 0 and stride(1 << 39, **step) == 0
            assert stride(1 << 40, **step) == code("LAYOUT") and stride(-1, **step) == code("LAYOUT")
            assert stride(1 << 26) == (0 if call is conv else code("LAYOUT")) and stride((1 << 26) - 1) == 0
            far = {"tokens": (1 << 24) - 1, "sequences": (1 << 24) - 1, "slots": 1 << 24, "seq_start": None}
            assert stride(1 << 30, **far) == code("LAYOUT")     # ends past any memory

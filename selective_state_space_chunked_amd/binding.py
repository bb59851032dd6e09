"""ctypes binding of libssmscan.so (include/ssmscan.h).

Argument marshalling only: input tensors and caller-supplied outputs
(``out=``) are checked for device, dtype, shape and contiguity, missing
outputs and the workspace are allocated on the tensors' device (with
torch.empty, or with the allocator installed by ``set_allocator``), and every
step of the scan runs in the library's HIP kernels on torch's current stream.
There is no CPU fallback: tensors that are not on a GPU are rejected, and if
the library is missing or a call fails, this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssmscan.so")

SSM_F32, SSM_BF16 = 0, 1
SSM_EULER, SSM_ZOH = 0, 1
# roles of the strided views (ssm_layout)
(V_DELTA, V_X, V_A, V_BM, V_C, V_Y, V_GY, V_GDELTA, V_GX, V_R, V_PHI, V_U, V_LAM, V_THETA, V_CC, V_LOGITS,
 V_PD_D, V_PD_B, V_PD_C, V_DICT) = range(20)
V_COUNT = 20
SSM_REAL_SELECTIVE, SSM_REAL_DENSE, SSM_COMPLEX_SHARED, SSM_COMPLEX_DENSE, SSM_HEAD_SCALAR = 0, 1, 2, 3, 4
_COMPLEX_MODES = (SSM_COMPLEX_SHARED, SSM_COMPLEX_DENSE)
(SSM_OP_SCAN_FWD, SSM_OP_SCAN_BWD, SSM_OP_IMPULSE, SSM_OP_PD_FWD, SSM_OP_PD_BWD, SSM_OP_COMPLEX_RTRL,
 SSM_OP_OUTPUT_SENS, SSM_OP_SENS_ROWS, SSM_OP_CONV_FWD, SSM_OP_CONV_BWD, SSM_OP_TOKENS_CONV,
 SSM_OP_TOKENS_SCAN, SSM_OP_GATED_FWD, SSM_OP_GATED_BWD, SSM_OP_TOKENS_GATED, SSM_OP_GROUP_NORM_BWD) = range(16)
SSM_GATED_CHUNK = 128  # steps between the states that a gated recurrence keeps for its backward
SSM_CKPT8_BLOCK = 64   # steps of a row that share one scale of an 8-bit checkpoint

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


class Layout(ctypes.Structure):
    _fields_ = [("given", ctypes.c_uint64), ("stride", (ctypes.c_int64 * 4) * V_COUNT)]


class _Views:
    """The strides of the tensors of one call that are views (non-dense or broadcast)."""

    def __init__(self):
        self.lay = Layout()
        self.any = False

    def set(self, role, strides, dense):
        strides = tuple(int(v) for v in strides)
        if strides != tuple(int(v) for v in dense):
            self.lay.given |= 1 << role
            for i, v in enumerate(strides):
                self.lay.stride[role][i] = v
            self.any = True

    def ptr(self):
        return ctypes.pointer(self.lay) if self.any else None


def _dense_strides(shape):
    st, acc = [], 1
    for n in reversed(shape):
        st.append(acc)
        acc *= int(n)
    return tuple(reversed(st))


class ScanArgs(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("batch", _i64), ("channels", _i64), ("length", _i64), ("state", _i64), ("chunk_len", _i64),
                ("delta", _vp), ("x", _vp), ("A", _vp), ("Bm", _vp), ("a", _vp), ("b", _vp), ("C", _vp),
                ("r", _vp), ("phi", _vp), ("lam", _vp), ("theta", _vp), ("u", _vp), ("c", _vp), ("h0", _vp),
                ("delta_bias", _vp), ("delta_softplus", ctypes.c_int32), ("discretization", ctypes.c_int32),
                ("layout", ctypes.POINTER(Layout)), ("head_dim", _i64)]


class ScanFwdOut(ctypes.Structure):
    _fields_ = [("y", _vp), ("h_last", _vp), ("ckpt", _vp)]


class ScanBwdIn(ctypes.Structure):
    _fields_ = [("gy", _vp), ("gh_last", _vp), ("ckpt", _vp)]


class ScanGrads(ctypes.Structure):
    _fields_ = [("gdelta", _vp), ("gx", _vp), ("gA", _vp), ("gBm", _vp), ("ga", _vp), ("gb", _vp),
                ("gC", _vp), ("gu", _vp), ("gr", _vp), ("gphi", _vp), ("glam", _vp), ("gtheta", _vp),
                ("gc", _vp), ("gh0", _vp), ("gdelta_bias", _vp)]


class PDArgs(ctypes.Structure):
    _fields_ = [("batch", _i64), ("heads", _i64), ("length", _i64), ("state", _i64), ("dict_size", _i64),
                ("chunk_len", _i64), ("logits", _vp), ("sel", _vp), ("dict", _vp), ("d", _vp), ("b", _vp),
                ("C", _vp), ("h0", _vp), ("dtype", ctypes.c_int32), ("layout", ctypes.POINTER(Layout))]


class PDFwdOut(ctypes.Structure):
    _fields_ = [("y", _vp), ("sel", _vp), ("h_last", _vp), ("ckpt", _vp)]


class PDBwdIn(ctypes.Structure):
    _fields_ = [("gy", _vp), ("gh_last", _vp), ("ckpt", _vp), ("ste_logits", _vp), ("tau", ctypes.c_float)]


class PDGrads(ctypes.Structure):
    _fields_ = [("gd", _vp), ("gb", _vp), ("gC", _vp), ("gh0", _vp), ("glogits", _vp)]


class ConvArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("silu", ctypes.c_int32),
                ("batch", _i64), ("channels", _i64), ("length", _i64), ("width", _i64),
                ("x", _vp), ("x8", _vp), ("x8_scale", _vp), ("w", _vp), ("bias", _vp), ("init", _vp),
                ("layout", ctypes.POINTER(Layout))]


class ConvFwdOut(ctypes.Structure):
    _fields_ = [("y", _vp), ("last", _vp), ("x8", _vp), ("x8_scale", _vp)]


class ConvGrads(ctypes.Structure):
    _fields_ = [("gx", _vp), ("gw", _vp), ("gbias", _vp), ("ginit", _vp)]


class Ckpt8Args(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("batch", _i64), ("channels", _i64), ("length", _i64),
                ("layout", ctypes.POINTER(Layout))]


class TokensConvArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("silu", ctypes.c_int32),
                ("tokens", _i64), ("channels", _i64), ("width", _i64), ("sequences", _i64), ("slots", _i64),
                ("x", _vp), ("w", _vp), ("bias", _vp), ("seq_start", _vp), ("slot", _vp), ("fresh", _vp),
                ("pool", _vp), ("y", _vp), ("x_stride", _i64), ("y_stride", _i64), ("pool_stride", _i64)]


class TokensScanArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("delta_softplus", ctypes.c_int32),
                ("tokens", _i64), ("channels", _i64), ("state", _i64), ("sequences", _i64), ("slots", _i64),
                ("delta", _vp), ("x", _vp), ("A", _vp), ("Bm", _vp), ("C", _vp), ("delta_bias", _vp), ("skip", _vp),
                ("z", _vp), ("seq_start", _vp), ("slot", _vp), ("fresh", _vp), ("pool", _vp), ("y", _vp),
                ("delta_stride", _i64), ("x_stride", _i64), ("Bm_stride", _i64), ("C_stride", _i64),
                ("z_stride", _i64), ("y_stride", _i64), ("pool_stride", _i64)]


class GatedArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("power", ctypes.c_float),
                ("batch", _i64), ("channels", _i64), ("length", _i64),
                ("x", _vp), ("r", _vp), ("i", _vp), ("lam", _vp), ("r_bias", _vp), ("i_bias", _vp), ("h0", _vp),
                ("x_stride", _i64 * 2), ("r_stride", _i64 * 2), ("i_stride", _i64 * 2)]


class GatedFwdOut(ctypes.Structure):
    _fields_ = [("y", _vp), ("h_last", _vp), ("ckpt", _vp), ("y_stride", _i64 * 2)]


class GatedBwdIn(ctypes.Structure):
    _fields_ = [("gy", _vp), ("gh_last", _vp), ("ckpt", _vp), ("gy_stride", _i64 * 2)]


class GatedGrads(ctypes.Structure):
    _fields_ = [("gx", _vp), ("gr", _vp), ("gi", _vp), ("glam", _vp), ("gr_bias", _vp), ("gi_bias", _vp), ("gh0", _vp),
                ("gx_stride", _i64 * 2), ("gr_stride", _i64 * 2), ("gi_stride", _i64 * 2)]


class TokensGatedArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("power", ctypes.c_float),
                ("tokens", _i64), ("channels", _i64), ("sequences", _i64), ("slots", _i64),
                ("x", _vp), ("r", _vp), ("i", _vp), ("lam", _vp), ("r_bias", _vp), ("i_bias", _vp),
                ("seq_start", _vp), ("slot", _vp), ("fresh", _vp), ("pool", _vp), ("y", _vp),
                ("x_stride", _i64), ("r_stride", _i64), ("i_stride", _i64), ("y_stride", _i64), ("pool_stride", _i64)]


class GroupNormArgs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("silu", ctypes.c_int32), ("rows", _i64), ("channels", _i64), ("groups", _i64),
                ("x", _vp), ("z", _vp), ("w", _vp), ("bias", _vp), ("x_stride", _i64), ("z_stride", _i64),
                ("eps", ctypes.c_float)]


class GroupNormGrads(ctypes.Structure):
    _fields_ = [("gx", _vp), ("gz", _vp), ("gw", _vp), ("gbias", _vp), ("gx_stride", _i64), ("gz_stride", _i64)]


class TokensPack8Args(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("tokens", _i64), ("channels", _i64), ("x", _vp), ("x8", _vp),
                ("x8_scale", _vp), ("x_stride", _i64), ("x8_stride", _i64)]


class TokensMm8Args(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("tokens", _i64), ("inputs", _i64), ("outputs", _i64), ("x8", _vp),
                ("x8_scale", _vp), ("w8", _vp), ("w8_scale", _vp), ("bias", _vp), ("y", _vp), ("x8_stride", _i64),
                ("w8_stride", _i64), ("y_stride", _i64)]


_lib = None


def lib():
    """Load libssmscan.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library {LIB_PATH} is missing: run __graft_entry__.build() "
                               "(or python selective_state_space_chunked_amd/build.py)")
        L = ctypes.CDLL(LIB_PATH)
        L.ssm_workspace_bytes.argtypes = [ctypes.c_int, _vp, ctypes.POINTER(ctypes.c_size_t)]
        L.ssm_scan_fwd.argtypes = [ctypes.POINTER(ScanArgs), ctypes.POINTER(ScanFwdOut), _vp, ctypes.c_size_t, _vp]
        L.ssm_scan_fwd_noalloc.argtypes = [ctypes.POINTER(ScanArgs), ctypes.POINTER(ScanFwdOut), _vp]
        L.ssm_scan_bwd.argtypes = [ctypes.POINTER(ScanArgs), ctypes.POINTER(ScanBwdIn), ctypes.POINTER(ScanGrads),
                                   _vp, ctypes.c_size_t, _vp]
        L.ssm_impulse_sensitivity.argtypes = [ctypes.POINTER(ScanArgs), _i64, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.ssm_output_sensitivity.argtypes = [ctypes.POINTER(ScanArgs), _i64, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.ssm_sensitivity_rows.argtypes = [ctypes.POINTER(ScanArgs), _i64, ctypes.c_int32, _vp, _vp, ctypes.c_size_t,
                                           _vp]
        L.ssm_complex_rtrl.argtypes = [ctypes.POINTER(ScanArgs), _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.pd_scan_fwd.argtypes = [ctypes.POINTER(PDArgs), ctypes.POINTER(PDFwdOut), _vp, ctypes.c_size_t, _vp]
        L.pd_scan_bwd.argtypes = [ctypes.POINTER(PDArgs), ctypes.POINTER(PDBwdIn), ctypes.POINTER(PDGrads),
                                  _vp, ctypes.c_size_t, _vp]
        L.ssm_conv_fwd.argtypes = [_vp, _vp, _vp]
        L.ssm_conv_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.ssm_ckpt8_pack.argtypes = [_vp, _vp, _vp, _vp, _vp]
        L.ssm_ckpt8_unpack.argtypes = [_vp, _vp, _vp, _vp, _vp]
        L.ssm_tokens_conv.argtypes = [_vp, _vp]
        L.ssm_tokens_scan.argtypes = [_vp, _vp, ctypes.c_size_t, _vp]
        L.ssm_gated_fwd.argtypes = [_vp, _vp, _vp]
        L.ssm_gated_bwd.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.ssm_tokens_gated.argtypes = [_vp, _vp, ctypes.c_size_t, _vp]
        L.ssm_group_norm_fwd.argtypes = [_vp, _vp, _i64, _vp]
        L.ssm_group_norm_bwd.argtypes = [_vp, _vp, _i64, _vp, _vp, ctypes.c_size_t, _vp]
        L.ssm_tokens_pack8.argtypes = [_vp, _vp]
        L.ssm_tokens_mm8.argtypes = [_vp, _vp]
        L.ssm_status_string.restype = ctypes.c_char_p
        L.ssm_status_string.argtypes = [ctypes.c_int]
        L.ssm_last_error_detail.restype = ctypes.c_char_p
        L.ssm_abi_version.restype = ctypes.c_int
        _lib = L
    return _lib


# The convolution, checkpoint and packed-row functions go through a native module where a call's arguments are plain
# (csrc/pycall.cpp): single tokens and small layers are bound by what a call costs the host.  The module is built for one
# Python and torch; where it does not load, the path below takes every call, at more host time.
_pycall = None   # not loaded yet; False: not there


def _load_pycall():
    global _pycall
    L = lib()
    try:
        from . import _pycall as native
    except ImportError as e:
        warnings.warn(f"native calls not available ({e}): calls of the convolution, checkpoint and packed-row functions "
                      "take more host time", RuntimeWarning, stacklevel=4)
        _pycall = False
        return False
    native.bind(*(ctypes.cast(getattr(L, f), _vp).value for f in (
        "ssm_conv_fwd", "ssm_conv_bwd", "ssm_ckpt8_pack", "ssm_ckpt8_unpack", "ssm_tokens_conv", "ssm_tokens_scan",
        "ssm_gated_fwd", "ssm_gated_bwd", "ssm_tokens_gated", "ssm_group_norm_fwd", "ssm_group_norm_bwd",
        "ssm_tokens_pack8", "ssm_tokens_mm8", "ssm_workspace_bytes")))
    _pycall = native
    return native


class SSMError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{lib().ssm_status_string(status).decode()}: {detail}")
        self.status = status


def _check(rc: int):
    if rc != 0:
        raise SSMError(rc, lib().ssm_last_error_detail().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _need(t, name, dtype=None, shape=None, device=None, view=False):
    """Check a tensor argument.  ``view``: a strided view is accepted (any strides with the last dimension
    contiguous; the library takes its strides), otherwise the tensor must be contiguous."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if view:
        if t.dim() > 1 and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous (stride 1)")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


_allocator = None


def set_allocator(fn):
    """Install ``fn(shape, dtype, device, role) -> tensor`` for the outputs this module allocates
    (role "output") and the workspaces (role "workspace", uint8); None restores torch.empty.  A caller
    can route allocations to its own memory pool, or fill them with a sentinel (tests fill outputs
    with NaN, integers with -1, so an element a kernel never writes cannot pass as a result)."""
    global _allocator
    _allocator = fn


def _alloc(shape, dtype, device, role="output"):
    if _allocator is not None:
        t = _allocator(tuple(shape), dtype, device, role)
        if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != torch.device(device) \
                or not t.is_contiguous():
            raise ValueError(f"allocator returned {tuple(t.shape)} {t.dtype} on {t.device}, "
                             f"expected {tuple(shape)} {dtype} on {device}")
        return t
    return torch.empty(shape, dtype=dtype, device=device)


def _out(out, key, shape, dtype, device, view=False):
    """out[key]: the caller's tensor, checked like an input, or a new one of the given shape and dtype.
    ``view``: the caller's tensor may be a strided view (distinct elements, last dimension contiguous)."""
    if key in out and out[key] is not None:
        t = _need(out[key], f"out[{key!r}]", dtype, shape, device, view=view)
        if view and not _distinct(t):
            raise ValueError(f"out[{key!r}]: an output view needs distinct elements (no stride 0)")
        return t
    out[key] = _alloc(shape, dtype, device)
    return out[key]


def _distinct(t):
    """True when no two indices of t address the same element."""
    dims = sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1)
    span = 1
    for st, n in dims:
        if st < span:
            return False
        span += st * (n - 1)
    return True


def _on_gpu(device):
    """The library takes device pointers only: host tensors would reach the kernels as bad addresses."""
    if torch.device(device).type != "cuda":
        raise ValueError(f"tensors must be on a GPU device (got {device}); there is no CPU path")


def _workspace(op, args_ptr, device):
    n = ctypes.c_size_t(0)
    _check(lib().ssm_workspace_bytes(op, args_ptr, ctypes.byref(n)))
    if n.value == 0:
        return None, 0
    ws = _alloc((n.value + 256,), torch.uint8, device, "workspace")
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n.value], n.value


def n_chunks(L, chunk_len):
    return -(-L // chunk_len)


# ---------------------------------------------------------------------------
# diagonal scans
# ---------------------------------------------------------------------------
def _scan_args(mode, *, delta=None, x=None, A=None, Bm=None, a=None, b=None, C=None, r=None, phi=None, lam=None,
               theta=None, u=None, c=None, h0=None, delta_bias=None, delta_softplus=False, discretization=SSM_EULER,
               chunk_len=0):
    """Marshal the scan arguments.  Selective mode: with ``delta_bias`` (D,) or
    ``delta_softplus`` set, ``delta`` is the projection output z and the scan uses
    softplus(z + delta_bias) (or z + delta_bias); ``discretization`` SSM_ZOH selects the
    zero-order-hold input term.  Inputs may be strided views (slices, ``expand``): the
    selective delta, x, A, Bm, C (Bm, C either (B, L, N), shared by the channels, or
    (B, D, L, N), per channel unless expanded along D) and the complex r, phi, u, lam,
    theta, c; their strides go to the library."""
    vw = _Views()
    perd = False
    head_dim = 0
    if mode == SSM_HEAD_SCALAR:
        # delta (B,H,L) and A (H) one per head; x (B,H*P,L); Bm, C (B,L,N)
        _need(delta, "delta", view=True)
        Bsz, H, L = delta.shape
        st = delta.dtype
        if st not in (torch.float32, torch.bfloat16):
            raise TypeError("delta must be float32 or bfloat16")
        dev = delta.device
        _need(x, "x", view=True)
        if x.dim() != 3 or x.shape[0] != Bsz or x.shape[2] != L or x.shape[1] % H:
            raise ValueError(f"x has shape {tuple(x.shape)}; expected (B, H*P, L) with B={Bsz} H={H} L={L}")
        D = x.shape[1]
        head_dim = D // H
        N = Bm.shape[-1]
        _need(x, "x", st, (Bsz, D, L), dev, view=True)
        for nm, t, role in (("Bm", Bm, V_BM), ("C", C, V_C)):
            _need(t, nm, st, (Bsz, L, N), dev, view=True)
            vw.set(role, (t.stride(0), 0, t.stride(1), t.stride(2)), (L * N, 0, N, 1))
        _need(A, "A", torch.float32, (H,), dev, view=True)
        _need(h0, "h0", torch.float32, (Bsz, D, N), dev)
        vw.set(V_DELTA, delta.stride(), (H * L, L, 1))
        vw.set(V_X, x.stride(), (D * L, L, 1))
        vw.set(V_A, A.stride(), (1,))
        dt = SSM_BF16 if st == torch.bfloat16 else SSM_F32
    elif mode == SSM_REAL_SELECTIVE:
        _need(delta, "delta", view=True)
        Bsz, D, L = delta.shape
        N = A.shape[1]
        st = delta.dtype
        if st not in (torch.float32, torch.bfloat16):
            raise TypeError("delta must be float32 or bfloat16")
        dev = delta.device
        _need(x, "x", st, (Bsz, D, L), dev, view=True)
        for nm, t, role in (("Bm", Bm, V_BM), ("C", C, V_C)):
            if t is not None and t.dim() == 4:
                _need(t, nm, st, (Bsz, D, L, N), dev, view=True)
                vw.set(role, t.stride(), (L * N, 0, N, 1))
                perd = perd or (t.stride(1) != 0 and D > 1)
            else:
                _need(t, nm, st, (Bsz, L, N), dev, view=True)
                if t is not None:
                    vw.set(role, (t.stride(0), 0, t.stride(1), t.stride(2)), (L * N, 0, N, 1))
        _need(A, "A", torch.float32, (D, N), dev, view=True)
        _need(h0, "h0", torch.float32, (Bsz, D, N), dev)
        _need(delta_bias, "delta_bias", torch.float32, (D,), dev)
        vw.set(V_DELTA, delta.stride(), (D * L, L, 1))
        vw.set(V_X, x.stride(), (D * L, L, 1))
        vw.set(V_A, A.stride(), (N, 1))
        dt = SSM_BF16 if st == torch.bfloat16 else SSM_F32
    elif mode == SSM_REAL_DENSE:
        _need(a, "a", torch.float32)
        Bsz, D, L, N = a.shape
        dev = a.device
        _need(b, "b", torch.float32, (Bsz, D, L, N), dev)
        _need(C, "C", torch.float32, (Bsz, L, N), dev)
        _need(h0, "h0", torch.float32, (Bsz, D, N), dev)
        dt = SSM_F32
    elif mode == SSM_COMPLEX_DENSE:
        if a is None:
            raise ValueError("SSM_COMPLEX_DENSE needs the transitions a")
        _need(a, "a", torch.complex64)
        Bsz, D, L, N = a.shape
        dev = a.device
        _need(u, "u", torch.complex64, (Bsz, D, L, N), dev)
        _need(c, "c", torch.complex64, (D, N), dev)
        _need(h0, "h0", torch.complex64, (Bsz, D, N), dev)
        dt = SSM_F32
    else:
        # u: complex64 (B,H,L,M), or bfloat16 (B,H,L,M,2) holding (re, im) pairs; r, phi follow
        _need(u, "u", view=True)
        if u.dtype == torch.complex64:
            Bsz, D, L, N = u.shape
            st = torch.float32
            vw.set(V_U, u.stride(), _dense_strides(u.shape))
        elif u.dtype == torch.bfloat16 and u.dim() == 5 and u.shape[-1] == 2:
            Bsz, D, L, N = u.shape[:4]
            st = torch.bfloat16
            if u.stride(3) != 2 and N > 1:
                raise ValueError("u: the (re, im) pairs of the modes must be contiguous")
            if any(v % 2 for v in u.stride()[:3]):
                raise ValueError("u: strides must be whole (re, im) pairs")
            vw.set(V_U, tuple(v // 2 for v in u.stride()[:3]) + (1,), _dense_strides(u.shape[:4]))
        else:
            raise TypeError("u must be complex64 (B,H,L,M) or bfloat16 (B,H,L,M,2)")
        dev = u.device
        for nm, t, role in (("r", r, V_R), ("phi", phi, V_PHI)):
            _need(t, nm, st, (Bsz, D, L), dev, view=True)
            vw.set(role, t.stride(), (D * L, L, 1))
        for nm, t, role in (("lam", lam, V_LAM), ("theta", theta, V_THETA)):
            _need(t, nm, torch.float32, (D, N), dev, view=True)
            vw.set(role, t.stride(), (N, 1))
        _need(c, "c", torch.complex64, (D, N), dev, view=True)
        vw.set(V_CC, c.stride(), (N, 1))
        _need(h0, "h0", torch.complex64, (Bsz, D, N), dev)
        dt = SSM_BF16 if st == torch.bfloat16 else SSM_F32
    args = ScanArgs(mode=mode, dtype=dt, batch=Bsz, channels=D, length=L, state=N, chunk_len=chunk_len,
                    delta=_ptr(delta), x=_ptr(x), A=_ptr(A), Bm=_ptr(Bm), a=_ptr(a), b=_ptr(b), C=_ptr(C),
                    r=_ptr(r), phi=_ptr(phi), lam=_ptr(lam), theta=_ptr(theta), u=_ptr(u), c=_ptr(c),
                    h0=_ptr(h0), delta_bias=_ptr(delta_bias), delta_softplus=int(bool(delta_softplus)),
                    discretization=int(discretization), head_dim=head_dim)
    args._views = vw          # kept with the struct: the library reads it during the call
    args._perd = perd
    args.layout = vw.ptr()
    return args, (Bsz, D, L, N), dev


def _set_layout(args):
    args.layout = args._views.ptr()


def _stream_dtype(mode, tensors):
    """Element type of the per-step streams (y, gy and their gradients) of a call."""
    if mode in (SSM_REAL_SELECTIVE, SSM_HEAD_SCALAR):
        return tensors["delta"].dtype
    if mode == SSM_COMPLEX_SHARED and tensors["u"].dtype == torch.bfloat16:
        return torch.bfloat16
    return torch.float32


def _chunk(mode, chunk_len):
    if chunk_len:
        return chunk_len
    return {SSM_REAL_SELECTIVE: 256, SSM_HEAD_SCALAR: 64}.get(mode, 32)


def scan_fwd(mode, *, want_y=True, want_h_last=False, want_ckpt=False, chunk_len=0, out=None, **tensors):
    """Forward scan.  Returns dict with y, h_last, ckpt (those requested).

    ``out`` may hold preallocated output tensors (keys y, h_last, ckpt).
    """
    return _scan_fwd(mode, want_y, want_h_last, want_ckpt, chunk_len, out, tensors, noalloc=False)


def scan_fwd_noalloc(mode, *, want_y=True, want_h_last=False, want_ckpt=False, chunk_len=0, out=None, **tensors):
    """ssm_scan_fwd_noalloc: the forward scan with the library's static device scratch in place of a
    workspace (nothing is allocated when ``out`` holds every requested output).  Same results as
    scan_fwd; calls that overlap on one device race on the shared scratch."""
    return _scan_fwd(mode, want_y, want_h_last, want_ckpt, chunk_len, out, tensors, noalloc=True)


def _scan_fwd(mode, want_y, want_h_last, want_ckpt, chunk_len, out, tensors, noalloc):
    args, (Bsz, D, L, N), dev = _scan_args(mode, chunk_len=chunk_len, **tensors)
    out = dict(out or {})
    ydt = _stream_dtype(mode, tensors)
    sdt = torch.complex64 if mode in _COMPLEX_MODES else torch.float32
    nc = n_chunks(L, _chunk(mode, chunk_len))
    sel = mode in (SSM_REAL_SELECTIVE, SSM_HEAD_SCALAR)
    for k, want, shp, dt in (("y", want_y, (Bsz, D, L), ydt), ("h_last", want_h_last, (Bsz, D, N), sdt),
                             ("ckpt", want_ckpt, (Bsz, D, nc, N), sdt)):
        if want or out.get(k) is not None:
            _out(out, k, shp, dt, dev, view=sel and k == "y")
    if sel and out.get("y") is not None:
        args._views.set(V_Y, out["y"].stride(), (D * L, L, 1))
        _set_layout(args)
    _on_gpu(dev)
    o = ScanFwdOut(y=_ptr(out.get("y")), h_last=_ptr(out.get("h_last")), ckpt=_ptr(out.get("ckpt")))
    if noalloc:
        _check(lib().ssm_scan_fwd_noalloc(ctypes.byref(args), ctypes.byref(o), _stream(dev)))
        return out
    ws, nws = _workspace(SSM_OP_SCAN_FWD, ctypes.byref(args), dev)
    _check(lib().ssm_scan_fwd(ctypes.byref(args), ctypes.byref(o), _ptr(ws), nws, _stream(dev)))
    return out


_GRADS = {
    SSM_REAL_SELECTIVE: ("gdelta", "gx", "gA", "gBm", "gC", "gh0"),   # gdelta_bias on request
    SSM_HEAD_SCALAR: ("gdelta", "gx", "gA", "gBm", "gC", "gh0"),
    SSM_REAL_DENSE: ("ga", "gb", "gC", "gh0"),
    SSM_COMPLEX_SHARED: ("gu", "gr", "gphi", "glam", "gtheta", "gc", "gh0"),
    SSM_COMPLEX_DENSE: ("ga", "gu", "gc", "gh0"),
}


def scan_bwd(mode, *, gy, gh_last=None, ckpt=None, want=None, chunk_len=0, out=None, **tensors):
    """Backward scan.  ``want`` lists gradient names (default: all of the mode)."""
    args, (Bsz, D, L, N), dev = _scan_args(mode, chunk_len=chunk_len, **tensors)
    ydt = _stream_dtype(mode, tensors)
    sdt = torch.complex64 if mode in _COMPLEX_MODES else torch.float32
    sel = mode in (SSM_REAL_SELECTIVE, SSM_HEAD_SCALAR)
    _need(gy, "gy", ydt, (Bsz, D, L), dev, view=sel)
    _need(gh_last, "gh_last", sdt, (Bsz, D, N), dev)
    nc = n_chunks(L, _chunk(mode, chunk_len))
    _need(ckpt, "ckpt", sdt, (Bsz, D, nc, N), dev)
    want = tuple(want) if want is not None else _GRADS[mode]
    gbc = (Bsz, D, L, N) if args._perd else (Bsz, L, N)   # per-channel B_t, C_t: per-channel gradients
    shapes = {
        "gdelta": ((Bsz, D, L), ydt), "gx": ((Bsz, D, L), ydt), "gA": ((D, N), torch.float32),
        "gBm": (gbc, ydt), "gC": (gbc, ydt), "gh0": ((Bsz, D, N), sdt),
        "ga": ((Bsz, D, L, N), sdt), "gb": ((Bsz, D, L, N), torch.float32),
        "gu": (((Bsz, D, L, N), torch.complex64) if ydt == torch.float32 else ((Bsz, D, L, N, 2), ydt)),
        "gr": ((Bsz, D, L), ydt), "gphi": ((Bsz, D, L), ydt), "glam": ((D, N), torch.float32),
        "gtheta": ((D, N), torch.float32), "gc": ((D, N), torch.complex64),
        "gdelta_bias": ((D,), torch.float32),
    }
    if mode == SSM_HEAD_SCALAR:   # per-head step sizes and transitions
        H = tensors["delta"].shape[1]
        shapes["gdelta"] = ((Bsz, H, L), ydt)
        shapes["gA"] = ((H,), torch.float32)
    out = dict(out or {})
    def exists(k):
        return k in _GRADS[mode] or (k == "gdelta_bias" and mode == SSM_REAL_SELECTIVE)
    for k in set(want) | {k for k, v in out.items() if v is not None}:
        if not exists(k):
            raise ValueError(f"gradient {k} does not exist for mode {mode}")
        _out(out, k, *shapes[k], dev, view=sel and k in ("gdelta", "gx"))
    if sel:
        args._views.set(V_GY, gy.stride(), (D * L, L, 1))
        for k, role in (("gdelta", V_GDELTA), ("gx", V_GX)):
            if out.get(k) is not None:
                args._views.set(role, out[k].stride(), _dense_strides(out[k].shape))
        _set_layout(args)
    _on_gpu(dev)
    g = ScanGrads(**{f[0]: _ptr(out.get(f[0])) for f in ScanGrads._fields_})
    i = ScanBwdIn(gy=_ptr(gy), gh_last=_ptr(gh_last), ckpt=_ptr(ckpt))
    ws, nws = _workspace(SSM_OP_SCAN_BWD, ctypes.byref(args), dev)
    _check(lib().ssm_scan_bwd(ctypes.byref(args), ctypes.byref(i), ctypes.byref(g), _ptr(ws), nws, _stream(dev)))
    return out


def impulse_sensitivity(*, t_out=-1, want_y=True, chunk_len=0, out=None, **tensors):
    """s[b,d,t] = d y[b,d,t_out] / d x[b,d,t] of a selective real scan (and y)."""
    args, (Bsz, D, L, N), dev = _scan_args(SSM_REAL_SELECTIVE, chunk_len=chunk_len, **tensors)
    dt = tensors["delta"].dtype
    out = dict(out or {})
    _out(out, "s", (Bsz, D, L), dt, dev)
    if want_y or out.get("y") is not None:
        _out(out, "y", (Bsz, D, L), dt, dev)
    _on_gpu(dev)
    ws, nws = _workspace(SSM_OP_IMPULSE, ctypes.byref(args), dev)
    _check(lib().ssm_impulse_sensitivity(ctypes.byref(args), int(t_out), _ptr(out.get("y")), _ptr(out["s"]),
                                         _ptr(ws), nws, _stream(dev)))
    return out


def output_sensitivity(*, t_out=-1, want_y=False, want_s_x=True, chunk_len=0, out=None, **tensors):
    """d y[b,d,t_out] / d x[b,d,t] (s_x) and / d delta[b,d,t] (s_delta) of a selective real scan (and y)."""
    args, (Bsz, D, L, N), dev = _scan_args(SSM_REAL_SELECTIVE, chunk_len=chunk_len, **tensors)
    dt = tensors["delta"].dtype
    out = dict(out or {})
    for k, want in (("s_delta", True), ("s_x", want_s_x), ("y", want_y)):
        if want or out.get(k) is not None:
            _out(out, k, (Bsz, D, L), dt, dev)
    _on_gpu(dev)
    ws, nws = _workspace(SSM_OP_OUTPUT_SENS, ctypes.byref(args), dev)
    _check(lib().ssm_output_sensitivity(ctypes.byref(args), int(t_out), _ptr(out.get("y")), _ptr(out.get("s_x")),
                                        _ptr(out["s_delta"]), _ptr(ws), nws, _stream(dev)))
    return out


def sensitivity_rows(*, t_out0, rows, out=None, **tensors):
    """s[r,b,d,t] = d y[b,d,t_out0+r] / d x[b,d,t] for r < rows (rows 1..16) of a selective real scan."""
    args, (Bsz, D, L, N), dev = _scan_args(SSM_REAL_SELECTIVE, **tensors)
    dt = tensors["delta"].dtype
    shp = (int(rows), Bsz, D, L)
    s = _need(out, "out", dt, shp, dev) if out is not None else _alloc(shp, dt, dev)
    _on_gpu(dev)
    ws, nws = _workspace(SSM_OP_SENS_ROWS, ctypes.byref(args), dev)
    _check(lib().ssm_sensitivity_rows(ctypes.byref(args), int(t_out0), int(rows), _ptr(s), _ptr(ws), nws,
                                      _stream(dev)))
    return s


def complex_rtrl(*, gy, gh_last=None, want_y=True, chunk_len=0, out=None, **tensors):
    """Forward-mode (real-time recurrent) glam and gtheta of the complex mode (and y).

    Loss = sum_t gy_t y_t + <gh_last, h_{L-1}>; returns dict with glam, gtheta
    ((H, M) float32) and y ((B, H, L) float32) when ``want_y``.
    """
    args, (Bsz, H, L, M), dev = _scan_args(SSM_COMPLEX_SHARED, chunk_len=chunk_len, **tensors)
    ydt = _stream_dtype(SSM_COMPLEX_SHARED, tensors)
    _need(gy, "gy", ydt, (Bsz, H, L), dev)
    _need(gh_last, "gh_last", torch.complex64, (Bsz, H, M), dev)
    out = dict(out or {})
    for k in ("glam", "gtheta"):
        _out(out, k, (H, M), torch.float32, dev)
    if want_y or out.get("y") is not None:
        _out(out, "y", (Bsz, H, L), ydt, dev)
    _on_gpu(dev)
    ws, nws = _workspace(SSM_OP_COMPLEX_RTRL, ctypes.byref(args), dev)
    _check(lib().ssm_complex_rtrl(ctypes.byref(args), _ptr(gy), _ptr(gh_last), _ptr(out.get("y")),
                                  _ptr(out["glam"]), _ptr(out["gtheta"]), _ptr(ws), nws, _stream(dev)))
    return out


# ---------------------------------------------------------------------------
# PD scan
# ---------------------------------------------------------------------------
def _pd_args(*, logits=None, sel=None, dict, d, b, C, h0=None, chunk_len=0):
    """Streams (logits, d, b, C) are all float32 or all bfloat16 (the dtype of d).  logits, d, b, C and
    the dictionary may be strided views (a dictionary expanded along the heads is shared by them)."""
    _need(d, "d", view=True)
    st = d.dtype
    if st not in (torch.float32, torch.bfloat16):
        raise TypeError("d must be float32 or bfloat16")
    Bsz, H, L, N = d.shape
    dev = d.device
    K = dict.shape[1]
    vw = _Views()
    _need(dict, "dict", torch.int32, (H, K, N), dev, view=True)
    _need(logits, "logits", st, (Bsz, H, L, K), dev, view=True)
    _need(sel, "sel", torch.int32, (Bsz, H, L), dev)
    if logits is None and sel is None:
        raise ValueError("logits or sel is required")
    for nm, t in (("b", b), ("C", C)):
        _need(t, nm, st, (Bsz, H, L, N), dev, view=True)
    _need(h0, "h0", torch.float32, (Bsz, H, N), dev)
    for t, role in ((d, V_PD_D), (b, V_PD_B), (C, V_PD_C)):
        vw.set(role, t.stride(), (H * L * N, L * N, N, 1))
    if logits is not None:
        vw.set(V_LOGITS, logits.stride(), (H * L * K, L * K, K, 1))
    vw.set(V_DICT, dict.stride(), (K * N, N, 1))
    args = PDArgs(batch=Bsz, heads=H, length=L, state=N, dict_size=K, chunk_len=chunk_len,
                  logits=_ptr(logits), sel=_ptr(sel), dict=_ptr(dict), d=_ptr(d), b=_ptr(b), C=_ptr(C),
                  h0=_ptr(h0), dtype=SSM_BF16 if st == torch.bfloat16 else SSM_F32)
    args._views = vw
    args.layout = vw.ptr()
    return args, (Bsz, H, L, N, K), dev


def pd_scan_fwd(*, want_y=True, want_sel=True, want_h_last=False, want_ckpt=False, chunk_len=0, out=None,
                **tensors):
    args, (Bsz, H, L, N, K), dev = _pd_args(chunk_len=chunk_len, **tensors)
    nc = n_chunks(L, chunk_len or 64)
    out = dict(out or {})
    for k, want, shp, dt in (("y", want_y, (Bsz, H, L), tensors["d"].dtype),
                             ("sel", want_sel, (Bsz, H, L), torch.int32),
                             ("h_last", want_h_last, (Bsz, H, N), torch.float32),
                             ("ckpt", want_ckpt, (Bsz, H, nc, N), torch.float32)):
        if want or out.get(k) is not None:
            _out(out, k, shp, dt, dev)
    _on_gpu(dev)
    o = PDFwdOut(y=_ptr(out.get("y")), sel=_ptr(out.get("sel")), h_last=_ptr(out.get("h_last")),
                 ckpt=_ptr(out.get("ckpt")))
    ws, nws = _workspace(SSM_OP_PD_FWD, ctypes.byref(args), dev)
    _check(lib().pd_scan_fwd(ctypes.byref(args), ctypes.byref(o), _ptr(ws), nws, _stream(dev)))
    return out


def pd_scan_bwd(*, gy, gh_last=None, ckpt=None, want=("gd", "gb", "gC", "gh0"), ste_logits=None, tau=1.0,
                chunk_len=0, out=None, **tensors):
    """PD backward with the selection held fixed.  ``want`` may also name
    "glogits", the straight-through surrogate gradient of ``ste_logits``
    (B, H, L, K) through softmax(ste_logits / tau)."""
    args, (Bsz, H, L, N, K), dev = _pd_args(chunk_len=chunk_len, **tensors)
    st = tensors["d"].dtype
    _need(gy, "gy", st, (Bsz, H, L), dev)
    _need(gh_last, "gh_last", torch.float32, (Bsz, H, N), dev)
    nc = n_chunks(L, chunk_len or 64)
    _need(ckpt, "ckpt", torch.float32, (Bsz, H, nc, N), dev)
    _need(ste_logits, "ste_logits", st, (Bsz, H, L, K), dev)
    out = dict(out or {})
    shapes = {"gd": (Bsz, H, L, N), "gb": (Bsz, H, L, N), "gC": (Bsz, H, L, N), "gh0": (Bsz, H, N),
              "glogits": (Bsz, H, L, K)}
    for k in set(want) | {k for k, v in out.items() if v is not None}:
        if k not in shapes:
            raise ValueError(f"unknown PD gradient {k}")
        _out(out, k, shapes[k], torch.float32 if k == "gh0" else st, dev)
    _on_gpu(dev)
    g = PDGrads(**{f[0]: _ptr(out.get(f[0])) for f in PDGrads._fields_})
    i = PDBwdIn(gy=_ptr(gy), gh_last=_ptr(gh_last), ckpt=_ptr(ckpt), ste_logits=_ptr(ste_logits), tau=float(tau))
    ws, nws = _workspace(SSM_OP_PD_BWD, ctypes.byref(args), dev)
    _check(lib().pd_scan_bwd(ctypes.byref(args), ctypes.byref(i), ctypes.byref(g), _ptr(ws), nws, _stream(dev)))
    return out


# ---------------------------------------------------------------------------
# short causal convolution, 8-bit activation checkpoints
#
# A call whose tensors are plain goes through the native module; the functions
# here take the others (views, installed allocators, caller-supplied outputs of
# the convolution, tensors of another device than the current one) and name what
# is wrong with a call.  They check a tensor by one short predicate and pass their
# structs as packed bytes.
# ---------------------------------------------------------------------------
_STREAM = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}
_F32 = torch.float32
_CONV_ARGS = struct.Struct("@iiqqqqPPPPPPP")      # ConvArgs
_FOUR_PTRS = struct.Struct("@PPPP")               # ConvFwdOut, ConvGrads
_CKPT8_ARGS = struct.Struct("@i4xqqqP")           # Ckpt8Args
_TOKENS_CONV_ARGS = struct.Struct("@iiqqqqqPPPPPPPPqqq")            # TokensConvArgs
_TOKENS_SCAN_ARGS = struct.Struct("@iiqqqqqPPPPPPPPPPPPPqqqqqqq")   # TokensScanArgs
_GATED_ARGS = struct.Struct("@ifqqqPPPPPPPqqqqqq")                  # GatedArgs
_GATED_IO = struct.Struct("@PPPqq")                                 # GatedFwdOut, GatedBwdIn
_GATED_GRADS = struct.Struct("@PPPPPPPqqqqqq")                      # GatedGrads
_TOKENS_GATED_ARGS = struct.Struct("@ifqqqqPPPPPPPPPPPqqqqq")       # TokensGatedArgs
_GROUP_NORM_ARGS = struct.Struct("@iiqqqPPPPqqf4x")                 # GroupNormArgs
_GROUP_NORM_GRADS = struct.Struct("@PPPPqq")                        # GroupNormGrads
_TOKENS_PACK8_ARGS = struct.Struct("@i4xqqPPPqq")                   # TokensPack8Args
_TOKENS_MM8_ARGS = struct.Struct("@i4xqqqPPPPPPqqq")                # TokensMm8Args


def _stream_code(dtype, name):
    if dtype not in _STREAM:
        raise TypeError(f"{name} must be float32 or bfloat16")
    return _STREAM[dtype]


def _dense(t, name, dtype, shape, dev):
    """Address of a dense tensor of this type, shape and device; 0 for None."""
    if t is None:
        return 0
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _need(t, name, dtype, shape, dev)
    return t.data_ptr()


def _new(out, key, dtype, shape, dev):
    """Address of out[key]: the caller's dense tensor, or a new one."""
    t = out.get(key)
    if t is None:
        t = out[key] = torch.empty(shape, dtype=dtype, device=dev) if _allocator is None else _alloc(shape, dtype, dev)
        return t.data_ptr()
    return _dense(t, f"out[{key!r}]", dtype, shape, dev)


def _streams(views):
    """The layout of the (B, D, L) streams that are not dense: [(role, tensor), ..] -> Layout or None."""
    vw = None
    for role, t in views:
        if t is not None and not t.is_contiguous():
            vw = vw or _Views()
            vw.set(role, t.stride(), _dense_strides(t.shape))
    return vw.lay if vw is not None and vw.any else None


# torch.cuda.current_stream builds a Stream object on every call, which costs more than the rest of a launch here
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _launch(dev, fn, *args):
    """Calls the library on the tensors' device (it launches on the current one) and its current stream."""
    if dev.type != "cuda":
        _on_gpu(dev)
    cur = torch.cuda.current_device()
    if dev.index is None or dev.index == cur:
        rc = fn(*args, _raw_stream(cur))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev.index))
    if rc:
        _check(rc)


def _native(t):
    """The native calls and where they launch, (module, device, stream), for a call with tensor t; else None: outputs
    come from an installed allocator, t is no GPU tensor, or the native module does not load."""
    if _allocator is not None or not (isinstance(t, torch.Tensor) and t.is_cuda):
        return None
    m = _load_pycall() if _pycall is None else _pycall
    if not m:
        return None
    dev = torch.cuda.current_device()
    return m, dev, _raw_stream(dev)


def _done(r):
    """Whether a native call was made: raises the library's error, False where the arguments are for the path below."""
    if r is NotImplemented:
        return False
    if r.__class__ is int:
        _check(r)
    return True


def _need_ckpt8(ckpt8):
    x8, scale = ckpt8
    _need(x8, "x8", torch.int8)
    if x8 is None or x8.dim() != 3:
        raise ValueError("x8 must be (B, D, L)")
    Bsz, D, L = x8.shape
    _need(scale, "x8_scale", _F32, (Bsz, D, n_chunks(L, SSM_CKPT8_BLOCK)), x8.device)
    if scale is None:
        raise ValueError("x8_scale is required")
    return x8, scale


def _conv_args(x, ckpt8, w, bias, init, silu, st):
    """Sizes, type and device of a call, and its packed arguments once a layout is known.  The input is ``x``
    (B, D, L), a strided view or dense, or ``ckpt8`` = (x8, x8_scale)."""
    if (x is None) == (ckpt8 is None):
        raise ValueError("one of x and ckpt8 is the input")
    x8 = scale = 0
    if x is not None:
        if not (isinstance(x, torch.Tensor) and x.dim() == 3 and (x.is_contiguous() or x.shape[2] <= 1
                                                                  or x.stride(2) == 1)):
            _need(x, "x", view=True)
            if x.dim() != 3:
                raise ValueError(f"x has shape {tuple(x.shape)}; expected (B, D, L)")
        if st is not None and x.dtype is not st:
            raise TypeError(f"x has dtype {x.dtype}, expected {st}")
        shape, dev, st, xp = x.shape, x.device, x.dtype, x.data_ptr()
    else:
        q, sc = _need_ckpt8(ckpt8)
        shape, dev, xp, x8, scale = q.shape, q.device, 0, q.data_ptr(), sc.data_ptr()
        if st is None:
            raise TypeError("dtype is required with ckpt8")
    code = _stream_code(st, "x")
    Bsz, D, L = shape
    if not (isinstance(w, torch.Tensor) and w.dim() == 2 and w.shape[0] == D):
        raise ValueError(f"w must be (D, W) with D={D}")
    W = w.shape[1]
    wp = _dense(w, "w", _F32, (D, W), dev)
    bp = _dense(bias, "bias", _F32, (D,), dev)
    ip = _dense(init, "init", st, (Bsz, D, W - 1), dev)

    def packed(layout):
        return _CONV_ARGS.pack(code, 1 if silu else 0, Bsz, D, L, W, xp, x8, scale, wp, bp, ip,
                               0 if layout is None else ctypes.addressof(layout))

    return packed, shape, W, st, dev


def conv_fwd(*, x=None, ckpt8=None, w, bias=None, init=None, silu=False, want_y=True, want_last=False,
             want_ckpt8=False, dtype=None, out=None):
    """Short causal depthwise convolution, y = act(bias + sum_k w[:, k] e[..., t + k]) with e = (init | x).

    ``x`` (B, D, L) float32 or bfloat16, any batch and channel stride; ``w`` (D, W) float32, W in 2..4, its
    last column for the step itself; ``init`` (B, D, W-1) the inputs before step 0.  Returns a dict with y,
    last (the last W-1 inputs, what a following segment takes as ``init``) and x8, x8_scale (the 8-bit
    checkpoint of x), those requested.  ``ckpt8`` = (x8, x8_scale) takes the place of x, with ``dtype`` that
    of y: the convolution's output again from its checkpoint."""
    if not out and ckpt8 is None and dtype is None and (nat := _native(x)):
        m, di, stream = nat
        r = m.conv_fwd(di, stream, x, None, None, w, bias, init, silu, want_y, want_last, want_ckpt8)
        if _done(r):
            return {k: v for k, v in zip(("y", "last", "x8", "x8_scale"), r) if v is not None}
    packed, shape, W, st, dev = _conv_args(x, ckpt8, w, bias, init, silu, dtype)
    Bsz, D, L = shape
    out = dict(out) if out else {}
    y = last = x8 = scale = 0
    if want_ckpt8 or out.get("x8") is not None or out.get("x8_scale") is not None:
        if x is None:
            raise ValueError("a checkpoint is written from x")
        x8 = _new(out, "x8", torch.int8, (Bsz, D, L), dev)
        scale = _new(out, "x8_scale", _F32, (Bsz, D, n_chunks(L, SSM_CKPT8_BLOCK)), dev)
    if out.get("y") is not None:
        y = _out(out, "y", (Bsz, D, L), st, dev, view=True).data_ptr()
    elif want_y:
        y = _new(out, "y", st, (Bsz, D, L), dev)
    if want_last or out.get("last") is not None:
        last = _new(out, "last", st, (Bsz, D, W - 1), dev)
    lay = _streams(((V_X, x), (V_Y, out.get("y"))))
    _launch(dev, lib().ssm_conv_fwd, packed(lay), _FOUR_PTRS.pack(y, last, x8, scale))
    return out


_CONV_GRADS = ("gx", "gw", "gbias", "ginit")


@functools.lru_cache(maxsize=1024)
def _conv_bwd_bytes(Bsz, D, L, W):
    args = ConvArgs(dtype=SSM_F32, batch=Bsz, channels=D, length=L, width=W, x=256, w=256)   # sizes only
    n = ctypes.c_size_t(0)
    _check(lib().ssm_workspace_bytes(SSM_OP_CONV_BWD, ctypes.byref(args), ctypes.byref(n)))
    return n.value


def _scratch(n, dev):
    """A workspace of n bytes, 256-byte aligned: (tensor, address)."""
    if n == 0:
        return None, 0
    t = torch.empty((n + 256,), dtype=torch.uint8, device=dev) if _allocator is None else \
        _alloc((n + 256,), torch.uint8, dev, "workspace")
    p = t.data_ptr()
    return t, p + (-p) % 256


def conv_bwd(*, gy, x=None, ckpt8=None, w, bias=None, init=None, silu=False, glast=None, want=_CONV_GRADS, out=None):
    """Gradients of <gy, y> + <glast, last> of ``conv_fwd``, from its input or its input's 8-bit checkpoint
    (then those of the values the checkpoint stands for).  Returns a dict of the gradients named in ``want``."""
    if want is not _CONV_GRADS:
        want = tuple(want)
    if not out and (nat := _native(gy)) and (want is _CONV_GRADS or set(want) <= set(_CONV_GRADS)):
        m, di, stream = nat
        q, sc = ckpt8 if ckpt8 is not None else (None, None)
        r = m.conv_bwd(di, stream, gy, glast, x, q, sc, w, bias, init, silu, *[k in want for k in _CONV_GRADS])
        if _done(r):
            return {k: v for k, v in zip(_CONV_GRADS, r) if v is not None}
    if not isinstance(gy, torch.Tensor):
        raise ValueError("gy must be a torch.Tensor")
    packed, shape, W, st, dev = _conv_args(x, ckpt8, w, bias, init, silu, gy.dtype)
    Bsz, D, L = shape
    if gy.is_contiguous():
        gp = _dense(gy, "gy", st, shape, dev)
    else:
        gp = _need(gy, "gy", st, shape, dev, view=True).data_ptr()
    lp = _dense(glast, "glast", st, (Bsz, D, W - 1), dev)
    out = dict(out) if out else {}
    for k in (*want, *out):
        if k not in _CONV_GRADS:
            raise ValueError(f"unknown gradient {k}")
    gx = gw = gb = gi = 0
    if out.get("gx") is not None:
        gx = _out(out, "gx", shape, st, dev, view=True).data_ptr()
    elif "gx" in want:
        gx = _new(out, "gx", st, (Bsz, D, L), dev)
    if "gw" in want or out.get("gw") is not None:
        gw = _new(out, "gw", _F32, (D, W), dev)
    if "gbias" in want or out.get("gbias") is not None:
        gb = _new(out, "gbias", _F32, (D,), dev)
    if "ginit" in want or out.get("ginit") is not None:
        gi = _new(out, "ginit", st, (Bsz, D, W - 1), dev)
    lay = _streams(((V_X, x), (V_GY, gy), (V_GX, out.get("gx"))))
    args = packed(lay)
    if dev.type != "cuda":
        _on_gpu(dev)
    nws = _conv_bwd_bytes(Bsz, D, L, W)
    ws, wp = _scratch(nws, dev)
    _launch(dev, lib().ssm_conv_bwd, args, gp, lp, _FOUR_PTRS.pack(gx, gw, gb, gi), wp, nws)
    return out


def ckpt8_pack(x, *, out=None):
    """The 8-bit checkpoint of a stream x (B, D, L): a dict with x8 (B, D, L) int8 and x8_scale
    (B, D, ceil(L / 64)) float32, one scale for every 64 steps of a row."""
    if not out and (nat := _native(x)):
        m, di, stream = nat
        r = m.ckpt8_pack(di, stream, x)
        if _done(r):
            return {"x8": r[0], "x8_scale": r[1]}
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a torch.Tensor")
    _need(x, "x", view=True)
    code = _stream_code(x.dtype, "x")
    if x.dim() != 3:
        raise ValueError(f"x has shape {tuple(x.shape)}; expected (B, D, L)")
    Bsz, D, L = x.shape
    dev = x.device
    out = dict(out) if out else {}
    x8 = _new(out, "x8", torch.int8, (Bsz, D, L), dev)
    scale = _new(out, "x8_scale", _F32, (Bsz, D, n_chunks(L, SSM_CKPT8_BLOCK)), dev)
    lay = _streams(((V_X, x),))
    args = _CKPT8_ARGS.pack(code, Bsz, D, L, 0 if lay is None else ctypes.addressof(lay))
    _launch(dev, lib().ssm_ckpt8_pack, args, x.data_ptr(), x8, scale)
    return out


def ckpt8_unpack(x8, x8_scale, *, dtype=torch.float32, out=None):
    """The stream (B, D, L) of ``dtype`` that an 8-bit checkpoint stands for (what ``scan_bwd`` and other
    readers of whole streams take)."""
    if out is None and dtype in _STREAM and (nat := _native(x8)):
        m, di, stream = nat
        r = m.ckpt8_unpack(di, stream, x8, x8_scale, dtype is torch.bfloat16)
        if _done(r):
            return r
    x8, x8_scale = _need_ckpt8((x8, x8_scale))
    code = _stream_code(dtype, "dtype")
    Bsz, D, L = x8.shape
    dev = x8.device
    y = {"y": out}
    if out is None:
        _new(y, "y", dtype, (Bsz, D, L), dev)
    else:
        _out(y, "y", (Bsz, D, L), dtype, dev, view=True)
    y = y["y"]
    lay = _streams(((V_Y, y),))
    args = _CKPT8_ARGS.pack(code, Bsz, D, L, 0 if lay is None else ctypes.addressof(lay))
    _launch(dev, lib().ssm_ckpt8_unpack, args, x8.data_ptr(), x8_scale.data_ptr(), y.data_ptr())
    return y


# ---------------------------------------------------------------------------
# packed rows: serving forms with pools of states
# ---------------------------------------------------------------------------
def _rows(t, name, dtype, T, D, dev):
    """A matrix of rows: (address, row stride); rows contiguous, any stride from one to the next."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 2 and t.device == dev:
        r, c = t.shape
        if r == T and c == D:
            s0, s1 = t.stride()
            if s1 == 1 or D <= 1 or T == 0:
                return t.data_ptr(), s0
    if t is None:
        raise ValueError(f"{name} is required")
    _need(t, name, dtype, (T, D), dev, view=True)
    return t.data_ptr(), t.stride(0)


def _y_rows(out, dtype, T, D, dev):
    y = out.get("y")
    if y is None:
        return _new(out, "y", dtype, (T, D), dev), D
    p, s = _rows(y, "out['y']", dtype, T, D, dev)
    if T > 1 and s < D:
        raise ValueError("out['y']: an output view needs distinct elements (no stride 0)")
    return p, s


def _sequences(T, pool, inner, pool_dtype, dev, seq_start, slot, fresh):
    """Checks of the sequences of a call; (sequences, slots, pool stride, addresses of seq_start, slot, fresh)."""
    if not isinstance(pool, torch.Tensor) or pool.dim() != 3 or pool.shape[1:] != inner:
        raise ValueError(f"pool must be (slots, {inner[0]}, {inner[1]})")
    if pool.dtype is not pool_dtype:
        raise TypeError(f"pool has dtype {pool.dtype}, expected {pool_dtype}")
    if pool.device != dev:
        raise ValueError(f"pool is on {pool.device}, expected {dev}")
    st = pool.stride()
    if pool.numel() and (st[2] != 1 and inner[1] > 1 or st[1] != inner[1] and inner[0] > 1):
        raise ValueError("pool: every slot must be contiguous")
    S, start = T, 0
    if seq_start is not None:
        if not isinstance(seq_start, torch.Tensor) or seq_start.dim() != 1 or seq_start.shape[0] < 1:
            raise ValueError("seq_start must be (sequences + 1,)")
        S = seq_start.shape[0] - 1
        start = _dense(seq_start, "seq_start", torch.int32, (S + 1,), dev)
    sl = _dense(slot, "slot", torch.int32, (S,), dev)
    fr = 0
    if fresh is not None:
        if not isinstance(fresh, torch.Tensor):
            raise ValueError("fresh must be a torch.Tensor")
        if fresh.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"fresh has dtype {fresh.dtype}, expected torch.bool or torch.uint8")
        fr = _dense(fresh, "fresh", fresh.dtype, (S,), dev)
    return S, pool.shape[0], st[0], start, sl, fr


def _row_input(x):
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a torch.Tensor")
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}; expected (T, D)")
    T, D = x.shape
    return T, D, x.dtype, _stream_code(x.dtype, "x"), x.device


def tokens_conv(*, x, w, bias=None, silu=False, pool, seq_start=None, slot=None, fresh=None, out=None):
    """The convolution of ``conv_fwd`` over the packed rows x (T, D) of a batch of sequences.

    Sequence s owns rows seq_start[s] .. seq_start[s+1]-1 (``seq_start`` (S+1,) int32 on the device; None:
    one row a sequence).  ``pool`` (slots, D, W-1) holds each sequence's last W-1 inputs; sequence s begins
    with slot[s] (zeros where ``fresh``) and leaves its own there, in place.  A slot of -1 marks an empty
    place of the batch, which leaves its row as it was.  Returns a dict with y (T, D)."""
    if nat := _native(x):
        m, di, stream = nat
        y = out.get("y") if out else None
        r = m.tokens_conv(di, stream, x, w, bias, silu, seq_start, slot, fresh, pool, y)
        if _done(r):
            return dict(out) if y is not None else {**(out or {}), "y": r}
    T, D, st, code, dev = _row_input(x)
    xp, sx = _rows(x, "x", st, T, D, dev)
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[0] != D:
        raise ValueError(f"w must be (D, W) with D={D}")
    W = w.shape[1]
    wp = _dense(w, "w", _F32, (D, W), dev)
    bp = _dense(bias, "bias", _F32, (D,), dev)
    S, slots, spool, start, sl, fr = _sequences(T, pool, (D, W - 1), st, dev, seq_start, slot, fresh)
    out = dict(out) if out else {}
    yp, sy = _y_rows(out, st, T, D, dev)
    args = _TOKENS_CONV_ARGS.pack(code, 1 if silu else 0, T, D, W, S, slots, xp, wp, bp, start, sl, fr,
                                  pool.data_ptr(), yp, sx, sy, spool)
    _launch(dev, lib().ssm_tokens_conv, args)
    return out


@functools.lru_cache(maxsize=1024)
def _tokens_scan_bytes(T, D, N):
    # sizes only: the sequences do not change what the ranges of rows need
    args = TokensScanArgs(dtype=SSM_F32, tokens=T, channels=D, state=N, sequences=1, slots=1, seq_start=256,
                          delta_stride=D, x_stride=D, Bm_stride=N, C_stride=N, y_stride=D, pool_stride=D * N)
    n = ctypes.c_size_t(0)
    _check(lib().ssm_workspace_bytes(SSM_OP_TOKENS_SCAN, ctypes.byref(args), ctypes.byref(n)))
    return n.value


def tokens_scan(*, delta, x, A, Bm, C, skip=None, z=None, delta_bias=None, delta_softplus=False, pool,
                seq_start=None, slot=None, fresh=None, out=None):
    """The selective scan over the packed rows of a batch of sequences, with its layer's skip and gate:
    y = (C . h + skip * x) * z * sigmoid(z).

    ``delta``, ``x``, ``z`` (T, D) and ``Bm``, ``C`` (T, N) may be slices of wider rows; ``pool``
    (slots, D, N) float32 holds the states, in place; ``seq_start``, ``slot`` and ``fresh`` as in
    ``tokens_conv``; ``delta_bias`` and ``delta_softplus`` as in ``scan_fwd``.  Returns a dict with y (T, D)."""
    if nat := _native(x):
        m, di, stream = nat
        y = out.get("y") if out else None
        r = m.tokens_scan(di, stream, x, A, delta, Bm, C, z, skip, delta_bias, delta_softplus, seq_start, slot, fresh,
                          pool, y)
        if _done(r):
            return dict(out) if y is not None else {**(out or {}), "y": r}
    T, D, st, code, dev = _row_input(x)
    if not isinstance(A, torch.Tensor) or A.dim() != 2 or A.shape[0] != D:
        raise ValueError(f"A must be (D, N) with D={D}")
    N = A.shape[1]
    xp, sx = _rows(x, "x", st, T, D, dev)
    dp, sd = _rows(delta, "delta", st, T, D, dev)
    Bp, sB = _rows(Bm, "Bm", st, T, N, dev)
    Cp, sC = _rows(C, "C", st, T, N, dev)
    zp, sz = _rows(z, "z", st, T, D, dev) if z is not None else (0, 0)
    Ap = _dense(A, "A", _F32, (D, N), dev)
    kp = _dense(skip, "skip", _F32, (D,), dev)
    bp = _dense(delta_bias, "delta_bias", _F32, (D,), dev)
    S, slots, spool, start, sl, fr = _sequences(T, pool, (D, N), _F32, dev, seq_start, slot, fresh)
    out = dict(out) if out else {}
    yp, sy = _y_rows(out, st, T, D, dev)
    args = _TOKENS_SCAN_ARGS.pack(code, 1 if delta_softplus else 0, T, D, N, S, slots, dp, xp, Ap, Bp, Cp, bp, kp, zp,
                                  start, sl, fr, pool.data_ptr(), yp, sd, sx, sB, sC, sz, sy, spool)
    if dev.type != "cuda":
        _on_gpu(dev)
    nws = _tokens_scan_bytes(T, D, N) if seq_start is not None else 0
    ws, wp = _scratch(nws, dev)
    _launch(dev, lib().ssm_tokens_scan, args, wp, nws)
    return out


# ---------------------------------------------------------------------------
# gated linear recurrence
# ---------------------------------------------------------------------------
def _f32(v):
    """A real argument as a float32 can hold it (an infinity past its range: the library says what is wrong with it)."""
    v = float(v)
    return v if not abs(v) > 3.4028234663852886e38 else math.copysign(math.inf, v)


def _stream_of(t, name, dtype, shape, dev):
    """A (B, D, L) stream: (address, batch stride, channel stride); steps contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and (shape[2] <= 1 or t.stride(2) == 1 or t.is_contiguous())):
        if t is None:
            raise ValueError(f"{name} is required")
        _need(t, name, dtype, shape, dev, view=True)
    s = t.stride()
    return t.data_ptr(), s[0], s[1]


def _out_stream(out, key, want, dtype, shape, dev):
    """out[key], or a new stream where it is wanted; (0, 0, 0) for none."""
    if out.get(key) is None:
        if not want:
            return 0, 0, 0
        return _new(out, key, dtype, shape, dev), shape[1] * shape[2], shape[2]
    t = _out(out, key, shape, dtype, dev, view=True)
    return t.data_ptr(), t.stride(0), t.stride(1)


def _gated_args(x, r, i, lam, r_bias, i_bias, power, h0, st):
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a torch.Tensor")
    if x.dim() != 3:
        raise ValueError(f"x has shape {tuple(x.shape)}; expected (B, D, L)")
    if st is not None and x.dtype is not st:
        raise TypeError(f"x has dtype {x.dtype}, expected {st}")
    st, dev, shape = x.dtype, x.device, x.shape
    code = _stream_code(st, "x")
    Bsz, D, L = shape
    xp, *sx = _stream_of(x, "x", st, shape, dev)
    rp, *sr = _stream_of(r, "r", st, shape, dev)
    ip, *si = _stream_of(i, "i", st, shape, dev)
    if lam is None:
        raise ValueError("lam is required")
    lp, rb, ib = (_dense(t, n, _F32, (D,), dev) for t, n in ((lam, "lam"), (r_bias, "r_bias"), (i_bias, "i_bias")))
    hp = _dense(h0, "h0", _F32, (Bsz, D), dev)
    return _GATED_ARGS.pack(code, _f32(power), Bsz, D, L, xp, rp, ip, lp, rb, ib, hp, *sx, *sr, *si), shape, st, dev


def gated_fwd(*, x, r, i, lam, r_bias=None, i_bias=None, power=8.0, h0=None, want_y=True, want_h_last=False,
              want_ckpt=False, out=None):
    """Gated linear recurrence, h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t + i_bias) x_t with
    a_t = exp(-power * softplus(lam) * sigmoid(r_t + r_bias)) and y = h.

    ``x``, ``r``, ``i`` (B, D, L) float32 or bfloat16, any batch and channel stride; ``lam``, ``r_bias``, ``i_bias``
    (D,) and ``h0`` (B, D) float32.  Returns a dict with y, h_last (B, D) and ckpt (B, D, ceil(L / 128)), the states
    that ``gated_bwd`` begins from, those requested."""
    if not out and (nat := _native(x)):
        m, di, stream = nat
        t = m.gated_fwd(di, stream, x, r, i, lam, r_bias, i_bias, power, h0, want_y, want_h_last, want_ckpt)
        if _done(t):
            return {k: v for k, v in zip(("y", "h_last", "ckpt"), t) if v is not None}
    args, shape, st, dev = _gated_args(x, r, i, lam, r_bias, i_bias, power, h0, None)
    Bsz, D, L = shape
    out = dict(out) if out else {}
    y = _out_stream(out, "y", want_y, st, shape, dev)
    last = ckpt = 0
    if want_h_last or out.get("h_last") is not None:
        last = _new(out, "h_last", _F32, (Bsz, D), dev)
    if want_ckpt or out.get("ckpt") is not None:
        ckpt = _new(out, "ckpt", _F32, (Bsz, D, n_chunks(L, SSM_GATED_CHUNK)), dev)
    _launch(dev, lib().ssm_gated_fwd, args, _GATED_IO.pack(y[0], last, ckpt, *y[1:]))
    return out


_GATED_GRADS_OF = ("gx", "gr", "gi", "glam", "gr_bias", "gi_bias", "gh0")


@functools.lru_cache(maxsize=1024)
def _gated_bwd_bytes(Bsz, D, L):
    args = GatedArgs(dtype=SSM_F32, power=1.0, batch=Bsz, channels=D, length=L)   # sizes only
    for s in (args.x_stride, args.r_stride, args.i_stride):
        s[0], s[1] = D * L, L
    n = ctypes.c_size_t(0)
    _check(lib().ssm_workspace_bytes(SSM_OP_GATED_BWD, ctypes.byref(args), ctypes.byref(n)))
    return n.value


def gated_bwd(*, gy, x, r, i, lam, r_bias=None, i_bias=None, power=8.0, h0=None, gh_last=None, ckpt=None,
              want=_GATED_GRADS_OF, out=None):
    """Gradients of <gy, y> + <gh_last, h_last> of ``gated_fwd``; without ``ckpt`` its states are formed again first.
    Returns a dict of the gradients named in ``want``; those of biases that were not given are of biases of 0."""
    if want is not _GATED_GRADS_OF:
        want = tuple(want)
    if not out and (nat := _native(gy)) and (want is _GATED_GRADS_OF or set(want) <= set(_GATED_GRADS_OF)):
        m, di, stream = nat
        t = m.gated_bwd(di, stream, gy, gh_last, ckpt, x, r, i, lam, r_bias, i_bias, power, h0,
                        *[k in want for k in _GATED_GRADS_OF])
        if _done(t):
            return {k: v for k, v in zip(_GATED_GRADS_OF, t) if v is not None}
    if not isinstance(gy, torch.Tensor):
        raise ValueError("gy must be a torch.Tensor")
    args, shape, st, dev = _gated_args(x, r, i, lam, r_bias, i_bias, power, h0, gy.dtype)
    Bsz, D, L = shape
    g, *sg = _stream_of(gy, "gy", st, shape, dev)
    lp = _dense(gh_last, "gh_last", _F32, (Bsz, D), dev)
    cp = _dense(ckpt, "ckpt", _F32, (Bsz, D, n_chunks(L, SSM_GATED_CHUNK)), dev)
    out = dict(out) if out else {}
    for k in (*want, *out):
        if k not in _GATED_GRADS_OF:
            raise ValueError(f"unknown gradient {k}")
    streams = [_out_stream(out, k, k in want, st, shape, dev) for k in _GATED_GRADS_OF[:3]]
    par = [_new(out, k, _F32, (Bsz, D) if k == "gh0" else (D,), dev) if k in want or out.get(k) is not None else 0
           for k in _GATED_GRADS_OF[3:]]
    if dev.type != "cuda":
        _on_gpu(dev)
    nws = _gated_bwd_bytes(Bsz, D, L)
    ws, wp = _scratch(nws, dev)
    _launch(dev, lib().ssm_gated_bwd, args, _GATED_IO.pack(g, lp, cp, *sg),
            _GATED_GRADS.pack(*(s[0] for s in streams), *par, *(v for s in streams for v in s[1:])), wp, nws)
    return out


@functools.lru_cache(maxsize=1024)
def _tokens_gated_bytes(code, T, D, S):
    # sizes only
    args = TokensGatedArgs(dtype=code, power=1.0, tokens=T, channels=D, sequences=S, slots=S, seq_start=256,
                           x_stride=D, r_stride=D, i_stride=D, y_stride=D, pool_stride=D)
    n = ctypes.c_size_t(0)
    _check(lib().ssm_workspace_bytes(SSM_OP_TOKENS_GATED, ctypes.byref(args), ctypes.byref(n)))
    return n.value


def tokens_gated(*, x, r, i, lam, r_bias=None, i_bias=None, power=8.0, pool, seq_start=None, slot=None, fresh=None,
                 out=None):
    """The recurrence of ``gated_fwd`` over the packed rows of a batch of sequences.

    ``x``, ``r``, ``i`` (T, D) may be slices of wider rows; ``pool`` (slots, D) float32 holds the states, in place;
    ``seq_start``, ``slot`` and ``fresh`` as in ``tokens_conv``.  Returns a dict with y (T, D)."""
    if nat := _native(x):
        m, di, stream = nat
        y = out.get("y") if out else None
        t = m.tokens_gated(di, stream, x, r, i, lam, r_bias, i_bias, power, seq_start, slot, fresh, pool, y)
        if _done(t):
            return dict(out) if y is not None else {**(out or {}), "y": t}
    T, D, st, code, dev = _row_input(x)
    xp, sx = _rows(x, "x", st, T, D, dev)
    rp, sr = _rows(r, "r", st, T, D, dev)
    ip, si = _rows(i, "i", st, T, D, dev)
    if lam is None:
        raise ValueError("lam is required")
    lp, rb, ib = (_dense(t, n, _F32, (D,), dev) for t, n in ((lam, "lam"), (r_bias, "r_bias"), (i_bias, "i_bias")))
    if not isinstance(pool, torch.Tensor) or pool.dim() != 2 or pool.shape[1] != D:
        raise ValueError(f"pool must be (slots, {D})")
    S, slots, spool, start, sl, fr = _sequences(T, pool.unsqueeze(2), (D, 1), _F32, dev, seq_start, slot, fresh)
    out = dict(out) if out else {}
    yp, sy = _y_rows(out, st, T, D, dev)
    args = _TOKENS_GATED_ARGS.pack(code, _f32(power), T, D, S, slots, xp, rp, ip, lp, rb, ib, start, sl, fr, pool.data_ptr(),
                                   yp, sx, sr, si, sy, spool)
    if dev.type != "cuda":
        _on_gpu(dev)
    nws = _tokens_gated_bytes(code, T, D, S) if seq_start is not None else 0
    ws, wp = _scratch(nws, dev)
    _launch(dev, lib().ssm_tokens_gated, args, wp, nws)
    return out


# ---------------------------------------------------------------------------
# group norm of rows
# ---------------------------------------------------------------------------
def _norm_args(x, groups, w, bias, eps, silu, z, st):
    if not isinstance(x, torch.Tensor):
        raise ValueError("x must be a torch.Tensor")
    if x.dim() != 2:
        raise ValueError(f"x has shape {tuple(x.shape)}; expected (T, C)")
    if not isinstance(groups, int):
        raise TypeError("groups must be an int")
    if not -2**63 <= groups < 2**63:
        raise ValueError(f"groups={groups} is out of range")
    T, C = x.shape
    if st is not None and x.dtype is not st:
        raise TypeError(f"x has dtype {x.dtype}, expected {st}")
    st, dev = x.dtype, x.device
    code = _stream_code(st, "x")
    xp, sx = _rows(x, "x", st, T, C, dev)
    zp, sz = _rows(z, "z", st, T, C, dev) if z is not None else (0, 0)
    wp = _dense(w, "w", _F32, (C,), dev)
    bp = _dense(bias, "bias", _F32, (C,), dev)
    return _GROUP_NORM_ARGS.pack(code, 1 if silu else 0, T, C, groups, xp, zp, wp, bp, sx, sz, _f32(eps)), T, C, st, dev


def _out_rows(out, key, want, dtype, T, C, dev):
    """out[key], or new rows where they are wanted: (address, row stride); (0, 0) for none."""
    t = out.get(key)
    if t is None:
        return (_new(out, key, dtype, (T, C), dev), C) if want else (0, 0)
    p, s = _rows(t, f"out[{key!r}]", dtype, T, C, dev)
    if T > 1 and s < C:
        raise ValueError(f"out[{key!r}]: an output view needs distinct elements (no stride 0)")
    return p, s


def group_norm_fwd(*, x, groups, w=None, bias=None, eps=1e-5, silu=False, z=None, out=None):
    """Group norm of the rows x (T, C), channels last: y = act((x - mean) / sqrt(var + eps) * w + bias), times
    z * sigmoid(z) with a gate ``z`` (T, C); act is the identity, or with ``silu`` v * sigmoid(v).

    The statistics are those of one group (C / groups consecutive channels) of one row, in float32: a group's differences
    to its mean are to stay below 2^57 and var + eps at least 2^-126.  ``x`` and ``z`` may be slices of wider rows; ``w``,
    ``bias`` (C,) float32.  Returns a dict with y (T, C)."""
    if nat := _native(x):
        m, di, stream = nat
        y = out.get("y") if out else None
        t = m.group_norm_fwd(di, stream, x, groups, w, bias, eps, silu, z, y)
        if _done(t):
            return dict(out) if y is not None else {**(out or {}), "y": t}
    args, T, C, st, dev = _norm_args(x, groups, w, bias, eps, silu, z, None)
    out = dict(out) if out else {}
    yp, sy = _y_rows(out, st, T, C, dev)
    _launch(dev, lib().ssm_group_norm_fwd, args, yp, sy)
    return out


_NORM_GRADS = ("gx", "gz", "gw", "gbias")


@functools.lru_cache(maxsize=1024)
def _norm_bwd_bytes(code, T, C, groups):
    args = GroupNormArgs(dtype=code, rows=T, channels=C, groups=groups, x_stride=C)   # sizes only
    n = ctypes.c_size_t(0)
    _check(lib().ssm_workspace_bytes(SSM_OP_GROUP_NORM_BWD, ctypes.byref(args), ctypes.byref(n)))
    return n.value


def group_norm_bwd(*, gy, x, groups, w=None, bias=None, eps=1e-5, silu=False, z=None, want=None, out=None):
    """Gradients of <gy, y> of ``group_norm_fwd``: a dict of those named in ``want`` (by default gx, gw, gbias, and gz
    with a gate); the statistics are formed again from x."""
    want = tuple(want) if want is not None else _NORM_GRADS if z is not None else ("gx", "gw", "gbias")
    if not out and (nat := _native(gy)) and (want is _NORM_GRADS or set(want) <= set(_NORM_GRADS)):
        m, di, stream = nat
        t = m.group_norm_bwd(di, stream, gy, x, groups, w, bias, eps, silu, z, *[k in want for k in _NORM_GRADS])
        if _done(t):
            return {k: v for k, v in zip(_NORM_GRADS, t) if v is not None}
    if not isinstance(gy, torch.Tensor):
        raise ValueError("gy must be a torch.Tensor")
    args, T, C, st, dev = _norm_args(x, groups, w, bias, eps, silu, z, gy.dtype)
    gp, sg = _rows(gy, "gy", st, T, C, dev)
    out = dict(out) if out else {}
    for k in (*want, *out):
        if k not in _NORM_GRADS:
            raise ValueError(f"unknown gradient {k}")
    gx, sgx = _out_rows(out, "gx", "gx" in want, st, T, C, dev)
    gz, sgz = _out_rows(out, "gz", "gz" in want, st, T, C, dev)
    gw, gb = (_new(out, k, _F32, (C,), dev) if k in want or out.get(k) is not None else 0 for k in ("gw", "gbias"))
    if dev.type != "cuda":
        _on_gpu(dev)
    nws = _norm_bwd_bytes(_STREAM[st], T, C, groups)
    ws, wp = _scratch(nws, dev)
    _launch(dev, lib().ssm_group_norm_bwd, args, gp, sg, _GROUP_NORM_GRADS.pack(gx, gz, gw, gb, sgx, sgz), wp, nws)
    return out


# ---------------------------------------------------------------------------
# products in 8-bit integers
# ---------------------------------------------------------------------------
def tokens_pack8(x, *, out=None):
    """The rows x (T, K) in 8 bits: a dict with x8 (T, K) int8 and x8_scale (T,) float32, one scale a row."""
    if not out and (nat := _native(x)):
        m, di, stream = nat
        t = m.tokens_pack8(di, stream, x)
        if _done(t):
            return {"x8": t[0], "x8_scale": t[1]}
    T, K, st, code, dev = _row_input(x)
    xp, sx = _rows(x, "x", st, T, K, dev)
    out = dict(out) if out else {}
    qp, sq = _out_rows(out, "x8", True, torch.int8, T, K, dev)
    sp = _new(out, "x8_scale", _F32, (T,), dev)
    _launch(dev, lib().ssm_tokens_pack8, _TOKENS_PACK8_ARGS.pack(code, T, K, xp, qp, sp, sx, sq))
    return out


def tokens_mm8(*, x8, x8_scale, w8, w8_scale, bias=None, dtype=torch.bfloat16, out=None):
    """The product of rows in 8 bits with weights in 8 bits, y = (x8 @ w8.T) * x8_scale[:, None] * w8_scale + bias.

    ``x8`` (T, K) int8 with ``x8_scale`` (T,), as ``tokens_pack8`` makes them; ``w8`` (N, K) int8 with ``w8_scale`` (N,);
    ``bias`` (N,) float32.  The sums are exact.  Returns a dict with y (T, N) of ``dtype`` (float32 or bfloat16)."""
    if dtype in _STREAM and (nat := _native(x8)):
        m, di, stream = nat
        y = out.get("y") if out else None
        t = m.tokens_mm8(di, stream, x8, x8_scale, w8, w8_scale, bias, dtype is torch.bfloat16, y)
        if _done(t):
            return dict(out) if y is not None else {**(out or {}), "y": t}
    for t, name in ((x8, "x8"), (w8, "w8")):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch.Tensor")
        if t.dim() != 2:
            raise ValueError(f"{name} has shape {tuple(t.shape)}; expected two dimensions")
    T, K = x8.shape
    N, dev = w8.shape[0], x8.device
    code = _stream_code(dtype, "dtype")
    xp, sx = _rows(x8, "x8", torch.int8, T, K, dev)
    wp, sw = _rows(w8, "w8", torch.int8, N, K, dev)
    if x8_scale is None or w8_scale is None:
        raise ValueError("x8_scale and w8_scale are required")
    xs = _dense(x8_scale, "x8_scale", _F32, (T,), dev)
    ws = _dense(w8_scale, "w8_scale", _F32, (N,), dev)
    bp = _dense(bias, "bias", _F32, (N,), dev)
    out = dict(out) if out else {}
    yp, sy = _y_rows(out, dtype, T, N, dev)
    _launch(dev, lib().ssm_tokens_mm8, _TOKENS_MM8_ARGS.pack(code, T, K, N, xp, xs, wp, ws, bp, yp, sx, sw, sy))
    return out

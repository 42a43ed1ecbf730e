"""Binding of the layer operators of libgdn.so (include/gdn.h): the short causal convolution, the
selective state space scan, the linear attention with a decay, the group norm, the norms around a block
and the projection. Argument marshalling only, as in binding.py.

Inputs that the header gives a row stride may be slices of a wider tensor along the last dimension
(x[..., :C] of a contiguous tensor); everything else must be contiguous. A call with stream=s is the
call under torch.cuda.stream(s).
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from .binding import (GDN_OK, INT_MAX, GdnError, _dtype_code, _int_sizes, _other_device, _require_cuda, _under,
                      load_library)
from .binding import _check as _check_in_words

GDN_ACT_NONE, GDN_ACT_SILU, GDN_ACT_GELU = 0, 1, 2
_ACTS = {"none": GDN_ACT_NONE, "silu": GDN_ACT_SILU, "gelu": GDN_ACT_GELU}
_SCAN_TILE = 16   # steps between the scan's checkpoints

_VP, _SZ, _LL, _I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_int


class GdnConvShape(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("C", _I), ("W", _I), ("act", _I), ("dtype", _I), ("ldx", _LL)]


class GdnScanShape(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("C", _I), ("N", _I), ("G", _I), ("dtype", _I), ("ldu", _LL), ("lddt", _LL),
                ("ldz", _LL), ("ldB", _LL), ("ldC", _LL)]


class GdnNormShape(ctypes.Structure):
    _fields_ = [("M", _I), ("G", _I), ("D", _I), ("act", _I), ("center", _I), ("dtype", _I), ("eps", ctypes.c_float),
                ("ldx", _LL), ("ldz", _LL)]


class GdnLinearShape(ctypes.Structure):
    _fields_ = [("M", _I), ("N", _I), ("K", _I), ("act", _I), ("dtype", _I), ("ldx", _LL), ("ldw", _LL), ("ldres", _LL)]


class GdnLinattnShape(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("Hk", _I), ("Hv", _I), ("Dk", _I), ("Dv", _I), ("dtype", _I), ("ldq", _LL), ("ldk", _LL),
                ("ldv", _LL)]


class GdnResnormShape(ctypes.Structure):
    _fields_ = [("M", _I), ("D", _I), ("gate_rows", _I), ("act", _I), ("post", _I), ("pre", _I), ("dtype", _I), ("eps", ctypes.c_float),
                ("ldx", _LL), ("ldh", _LL), ("ldz", _LL)]


_declared = None


def _library():
    """libgdn.so with the signatures of the layer operators declared."""
    global _declared
    if _declared is not None:
        return _declared
    lib = load_library()
    P = ctypes.POINTER
    for name, shape, args in (
            ("gdn_conv_fwd", GdnConvShape, [_VP] * 8), ("gdn_conv_bwd", GdnConvShape, [_VP] * 12 + [_SZ, _VP]),
            ("gdn_scan_fwd", GdnScanShape, [_VP] * 13 + [_SZ, _VP, _SZ, _VP]),
            ("gdn_scan_bwd", GdnScanShape, [_VP] * 10 + [_SZ] + [_VP] * 12 + [_SZ, _VP]),
            ("gdn_norm_fwd", GdnNormShape, [_VP] * 7), ("gdn_norm_bwd", GdnNormShape, [_VP] * 11 + [_SZ, _VP]),
            ("gdn_linear_fwd", GdnLinearShape, [_VP] * 7 + [_SZ, _VP]),
            ("gdn_linear_bwd", GdnLinearShape, [_VP] * 8 + [_SZ, _VP]),
            ("gdn_linattn_fwd", GdnLinattnShape, [_VP] * 9 + [_SZ, _VP]),
            ("gdn_linattn_bwd", GdnLinattnShape, [_VP] * 13 + [_SZ, _VP]),
            ("gdn_resnorm_fwd", GdnResnormShape, [_VP] * 10), ("gdn_resnorm_bwd", GdnResnormShape, [_VP] * 16 + [_SZ, _VP])):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, [P(shape)] + args
    for name, shape in (("gdn_conv_bwd_workspace_bytes", GdnConvShape), ("gdn_scan_ckpt_bytes", GdnScanShape),
                        ("gdn_scan_fwd_workspace_bytes", GdnScanShape), ("gdn_scan_bwd_workspace_bytes", GdnScanShape),
                        ("gdn_norm_bwd_workspace_bytes", GdnNormShape),
                        ("gdn_linear_fwd_workspace_bytes", GdnLinearShape),
                        ("gdn_linear_bwd_workspace_bytes", GdnLinearShape),
                        ("gdn_linattn_fwd_workspace_bytes", GdnLinattnShape),
                        ("gdn_linattn_bwd_workspace_bytes", GdnLinattnShape),
                        ("gdn_resnorm_bwd_workspace_bytes", GdnResnormShape)):
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_size_t, [P(shape)]
    _declared = lib
    return lib


def _act(act):
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError(f"act is {act!r}, expected one of {sorted(_ACTS)}") from None


def _at(t):
    return None if t is None else t.data_ptr()


def _stream_of(device):
    """binding._stream"""
    index = device.index
    if index != _current_device():
        raise _other_device(device, _current_device())
    return _raw_stream(index)


def _type(t):
    return 1 if t.dtype is torch.bfloat16 else _dtype_code(t)


def _check(name, t, shape, dtype, device):
    """binding._check, whose comparisons in words run only for a tensor that one of these refuses: a
    single-token call is shorter than its checks otherwise."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _check_in_words(name, t, shape, dtype, device)


def _rows(name, t, shape, dtype, device, inner=1):
    """Row stride (0: packed) of a tensor whose last `inner` dimensions are packed and whose leading
    ones follow each other at one stride, as a slice of a contiguous tensor along its last dimension."""
    if t.is_contiguous() and t.shape == shape and t.dtype is dtype and t.device == device:
        return 0
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    width, packed = 1, True
    for size, stride in zip(reversed(t.shape[-inner:]), reversed(t.stride()[-inner:])):
        packed = packed and (size == 1 or stride == width)
        width *= size
    ld, rows = None, 1
    for size, stride in zip(reversed(t.shape[:-inner]), reversed(t.stride()[:-inner])):
        if size == 1:
            continue
        if ld is None and stride % rows == 0:
            ld = stride // rows
        packed = packed and ld is not None and stride == ld * rows
        rows *= size
    if not packed or (ld is not None and ld < width):
        raise ValueError(f"{name} must be contiguous, or a slice of a contiguous tensor along its last dimension")
    return 0 if ld is None else ld


def _scratch(name, t, need, device):
    """The caller's buffer, checked, or a new one for this call (None where nothing is needed)."""
    if t is None:
        return _empty(need, dtype=torch.uint8, device=device) if need else None
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    return t


def _size(t):
    return 0 if t is None else t.numel() * t.element_size()


def _raise(name, rc):
    raise GdnError(name, rc, _library())


# A single token's step takes the GPU a few microseconds, less than a Python call with this many
# arguments: the code below looks up, converts and calls no more than it has to.
_empty, _empty_like, _byref = torch.empty, torch.empty_like, ctypes.byref
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


# A shape structure holds sizes alone, which a program repeats; the library only reads it.
_linattn_shape, _resnorm_shape = lru_cache(256)(GdnLinattnShape), lru_cache(256)(GdnResnormShape)


def _new_like(t):
    """A packed tensor of t's shape and type."""
    return _empty_like(t) if t.is_contiguous() else _empty(t.shape, dtype=t.dtype, device=t.device)


# ------------------------------------------------------------------- short causal convolution
def _conv_args(x, w, bias, s0, lens, act):
    B, T, C = x.shape
    W = w.shape[-1]
    dev, dt = x.device, x.dtype
    if x.numel() > INT_MAX or W > INT_MAX:
        _int_sizes("gdn_conv", B, T, C, W)
    ld = _rows("x", x, (B, T, C), dt, dev)
    _check("w", w, (C, W), _F32, dev)
    if bias is not None:
        _check("bias", bias, (C,), _F32, dev)
    if s0 is not None:
        _check("s0", s0, (B, W - 1, C), dt, dev)
    if lens is not None:
        _check("lens", lens, (B,), _I32, dev)
    return GdnConvShape(B, T, C, W, _act(act), _type(x), ld), B, T, C, W


def gdn_conv_fwd(x, w, bias=None, s0=None, lens=None, *, act="silu", y=None, s_T=None, want_s_T=True, stream=None):
    """y, s_T = gdn_conv_fwd(x, w[, bias, s0, lens]) on CUDA tensors (see include/gdn.h): the short
    causal convolution of x [B, T, C] with taps w [C, W] and an activation ("silu" or "none"); s0 and
    s_T [B, W-1, C] are the carried inputs (with T = 1, s_T may be s0: updated in place)."""
    if stream is not None:
        return _under(stream, gdn_conv_fwd, locals())
    lib = _library()
    shape, B, T, C, W = _conv_args(x, w, bias, s0, lens, act)
    dev, dt = x.device, x.dtype
    if y is not None:
        _check("y", y, (B, T, C), dt, dev)
    if s_T is not None:
        _check("s_T", s_T, (B, W - 1, C), dt, dev)
    if not x.is_cuda:
        _require_cuda(x)
    if y is None:
        y = _new_like(x)
    if s_T is None and want_s_T:
        s_T = _empty((B, W - 1, C), dtype=dt, device=dev) if s0 is None else _empty_like(s0)
    rc = lib.gdn_conv_fwd(_byref(shape), x.data_ptr(), w.data_ptr(), _at(bias), _at(s0), _at(lens), _at(y), _at(s_T), _stream_of(dev))
    if rc:
        _raise("gdn_conv_fwd", rc)
    return y, s_T


def gdn_conv_bwd_workspace_bytes(shape: GdnConvShape) -> int:
    return _library().gdn_conv_bwd_workspace_bytes(ctypes.byref(shape))


def gdn_conv_bwd(x, w, dy, bias=None, s0=None, lens=None, ds_T=None, *, act="silu", workspace=None, want_ds0=True, stream=None):
    """dict(dx, dw, dbias, ds0) = gdn_conv_bwd(x, w, dy, ...) for the inputs of gdn_conv_fwd; dw and
    dbias are float32. ds0 is None with want_ds0=False."""
    if stream is not None:
        return _under(stream, gdn_conv_bwd, locals())
    lib = _library()
    shape, B, T, C, W = _conv_args(x, w, bias, s0, lens, act)
    dev, dt = x.device, x.dtype
    _check("dy", dy, (B, T, C), dt, dev)
    if ds_T is not None:
        _check("ds_T", ds_T, (B, W - 1, C), dt, dev)
    if not x.is_cuda:
        _require_cuda(x)
    workspace = _scratch("workspace", workspace, lib.gdn_conv_bwd_workspace_bytes(_byref(shape)), dev)
    out = {"dx": _empty_like(dy), "dw": _empty_like(w),
           "dbias": _empty((C,), dtype=_F32, device=dev),
           "ds0": _empty((B, W - 1, C), dtype=dt, device=dev) if want_ds0 else None}
    rc = lib.gdn_conv_bwd(_byref(shape), x.data_ptr(), w.data_ptr(), _at(bias), _at(s0), _at(lens), dy.data_ptr(), _at(ds_T), _at(out["dx"]),
         _at(out["dw"]), _at(out["dbias"]), _at(out["ds0"]), _at(workspace), _size(workspace), _stream_of(dev))
    if rc:
        _raise("gdn_conv_bwd", rc)
    return out


# ------------------------------------------------------------------ selective state space scan
def _scan_args(u, dt, A_log, B, C, D, dt_bias, z, lens):
    Bn, T, Cn = u.shape
    G, N = B.shape[-2:]
    dev, ty = u.device, u.dtype
    if u.numel() > INT_MAX or B.numel() > INT_MAX:
        _int_sizes("gdn_scan", Bn, T, Cn, N, G)
    ldu, lddt = _rows("u", u, (Bn, T, Cn), ty, dev), _rows("dt", dt, (Bn, T, Cn), ty, dev)
    ldz = 0 if z is None else _rows("z", z, (Bn, T, Cn), ty, dev)
    ldB, ldC = _rows("B", B, (Bn, T, G, N), ty, dev, 2), _rows("C", C, (Bn, T, G, N), ty, dev, 2)
    _check("A_log", A_log, (Cn, N), _F32, dev)
    if D is not None:
        _check("D", D, (Cn,), _F32, dev)
    if dt_bias is not None:
        _check("dt_bias", dt_bias, (Cn,), _F32, dev)
    if lens is not None:
        _check("lens", lens, (Bn,), _I32, dev)
    return GdnScanShape(Bn, T, Cn, N, G, _type(u), ldu, lddt, ldz, ldB, ldC), Bn, T, Cn, N


def gdn_scan_ckpt_bytes(shape: GdnScanShape) -> int:
    return _library().gdn_scan_ckpt_bytes(ctypes.byref(shape))


def gdn_scan_fwd_workspace_bytes(shape: GdnScanShape) -> int:
    return _library().gdn_scan_fwd_workspace_bytes(ctypes.byref(shape))


def gdn_scan_bwd_workspace_bytes(shape: GdnScanShape) -> int:
    return _library().gdn_scan_bwd_workspace_bytes(ctypes.byref(shape))


def _scan_ckpt_shape(Bn, T, Cn, N):
    return (Bn, -(-T // _SCAN_TILE), Cn, N)


def gdn_scan_fwd(u, dt, A_log, B, C, D=None, dt_bias=None, z=None, h0=None, lens=None, *, y=None, h_T=None, ckpt=None,
                 workspace=None, want_h_T=True, want_ckpt=False, stream=None):
    """y, h_T, ckpt = gdn_scan_fwd(u, dt, A_log, B, C, ...) on CUDA tensors (see include/gdn.h): the
    selective state space scan of u [B, T, C] with steps dt, state inputs and outputs B, C [B, T, G, N]
    and gate z. ckpt [B, ceil(T / 16), C, N] (want_ckpt=True) is what gdn_scan_bwd needs. With T = 1
    and no ckpt, h_T may be h0: the state updated in place."""
    if stream is not None:
        return _under(stream, gdn_scan_fwd, locals())
    lib = _library()
    shape, Bn, T, Cn, N = _scan_args(u, dt, A_log, B, C, D, dt_bias, z, lens)
    dev = u.device
    if h0 is not None:
        _check("h0", h0, (Bn, Cn, N), _F32, dev)
    if y is not None:
        _check("y", y, (Bn, T, Cn), u.dtype, dev)
    if h_T is not None:
        _check("h_T", h_T, (Bn, Cn, N), _F32, dev)
    if ckpt is not None:
        _check("ckpt", ckpt, _scan_ckpt_shape(Bn, T, Cn, N), _F32, dev)
    if not u.is_cuda:
        _require_cuda(u)
    if y is None:
        y = _new_like(u)
    if h_T is None and want_h_T:
        h_T = _empty((Bn, Cn, N), dtype=_F32, device=dev) if h0 is None else _empty_like(h0)
    if ckpt is None and want_ckpt:
        ckpt = _empty(_scan_ckpt_shape(Bn, T, Cn, N), dtype=_F32, device=dev)
    if workspace is not None or T > 1:                 # a single step needs none
        workspace = _scratch("workspace", workspace, lib.gdn_scan_fwd_workspace_bytes(ctypes.byref(shape)), dev)
    rc = lib.gdn_scan_fwd(_byref(shape), u.data_ptr(), dt.data_ptr(), A_log.data_ptr(), B.data_ptr(), C.data_ptr(), _at(D), _at(dt_bias), _at(z), _at(h0),
         _at(lens), _at(y), _at(h_T), _at(ckpt), _size(ckpt), _at(workspace), _size(workspace), _stream_of(dev))
    if rc:
        _raise("gdn_scan_fwd", rc)
    return y, h_T, ckpt


def gdn_scan_bwd(u, dt, A_log, B, C, ckpt, dy, D=None, dt_bias=None, z=None, lens=None, dh_T=None, *, workspace=None,
                 want_dh0=True, stream=None):
    """dict(du, ddt, dA_log, dB, dC, dD, ddt_bias, dz, dh0) = gdn_scan_bwd(...) for the inputs and the
    ckpt of gdn_scan_fwd. dD, ddt_bias and dz are None where their input was, dh0 with want_dh0=False."""
    if stream is not None:
        return _under(stream, gdn_scan_bwd, locals())
    lib = _library()
    shape, Bn, T, Cn, N = _scan_args(u, dt, A_log, B, C, D, dt_bias, z, lens)
    dev, ty = u.device, u.dtype
    _check("ckpt", ckpt, _scan_ckpt_shape(Bn, T, Cn, N), _F32, dev)
    _check("dy", dy, (Bn, T, Cn), ty, dev)
    if dh_T is not None:
        _check("dh_T", dh_T, (Bn, Cn, N), _F32, dev)
    if not u.is_cuda:
        _require_cuda(u)
    workspace = _scratch("workspace", workspace, lib.gdn_scan_bwd_workspace_bytes(ctypes.byref(shape)), dev)
    vec = lambda t: None if t is None else _empty_like(t)  # noqa: E731
    out = {"du": _empty_like(dy), "ddt": _empty_like(dy), "dA_log": _empty_like(A_log),
           "dB": _new_like(B), "dC": _new_like(C),
           "dD": vec(D), "ddt_bias": vec(dt_bias), "dz": None if z is None else _empty_like(dy),
           "dh0": _empty((Bn, Cn, N), dtype=_F32, device=dev) if want_dh0 else None}
    rc = lib.gdn_scan_bwd(_byref(shape), u.data_ptr(), dt.data_ptr(), A_log.data_ptr(), B.data_ptr(), C.data_ptr(), _at(D), _at(dt_bias), _at(z), _at(lens),
         _at(ckpt), _size(ckpt), dy.data_ptr(), _at(dh_T), _at(out["du"]), _at(out["ddt"]), _at(out["dA_log"]), _at(out["dB"]),
         _at(out["dC"]), _at(out["dD"]), _at(out["ddt_bias"]), _at(out["dz"]), _at(out["dh0"]), _at(workspace),
         _size(workspace), _stream_of(dev))
    if rc:
        _raise("gdn_scan_bwd", rc)
    return out


# ---------------------------------------------------------------------------------- group norm
def _norm_args(x, groups, w, b, z, act, eps, center):
    dev, dt = x.device, x.dtype
    C = x.shape[-1]
    if groups < 1 or C % groups != 0:
        raise ValueError(f"{C} channels do not split into {groups} groups")
    rows = x.numel() // max(C, 1)
    if x.numel() > INT_MAX:
        _int_sizes("gdn_norm", rows, groups, C // groups)
    ldx = _rows("x", x, x.shape, dt, dev)
    ldz = 0 if z is None else _rows("z", z, x.shape, dt, dev)
    if w is not None:
        _check("w", w, (C,), _F32, dev)
    if b is not None:
        _check("b", b, (C,), _F32, dev)
    return GdnNormShape(rows, groups, C // groups, _act(act), 1 if center else 0, _type(x), eps, ldx, ldz)


def gdn_norm_fwd(x, groups, w=None, b=None, z=None, *, act="silu", eps=1e-5, center=True, y=None, stats=None,
                 want_stats=True, stream=None):
    """y, stats = gdn_norm_fwd(x, groups[, w, b, z]) on CUDA tensors (see include/gdn.h): group norm
    over the channels (last dimension) of every row of x, times w plus b, then the activation, or with
    a gate z the product with act(z). center=False: root mean square. stats [..., groups, 2] is what
    gdn_norm_bwd needs."""
    if stream is not None:
        return _under(stream, gdn_norm_fwd, locals())
    lib = _library()
    shape = _norm_args(x, groups, w, b, z, act, eps, center)
    dev = x.device
    stats_shape = tuple(x.shape[:-1]) + (groups, 2)
    if y is not None:
        _check("y", y, x.shape, x.dtype, dev)
    if stats is not None:
        _check("stats", stats, stats_shape, _F32, dev)
    if not x.is_cuda:
        _require_cuda(x)
    if y is None:
        y = _new_like(x)
    if stats is None and want_stats:
        stats = _empty(stats_shape, dtype=_F32, device=dev)
    rc = lib.gdn_norm_fwd(_byref(shape), x.data_ptr(), _at(w), _at(b), _at(z), _at(y), _at(stats), _stream_of(dev))
    if rc:
        _raise("gdn_norm_fwd", rc)
    return y, stats


def gdn_norm_bwd_workspace_bytes(shape: GdnNormShape) -> int:
    return _library().gdn_norm_bwd_workspace_bytes(ctypes.byref(shape))


def gdn_norm_bwd(x, groups, stats, dy, w=None, b=None, z=None, *, act="silu", eps=1e-5, center=True, workspace=None,
                 stream=None):
    """dict(dx, dw, db, dz) = gdn_norm_bwd(x, groups, stats, dy[, w, b, z]) for the inputs and stats of
    gdn_norm_fwd; dw, db (float32) and dz are None where their input was."""
    if stream is not None:
        return _under(stream, gdn_norm_bwd, locals())
    lib = _library()
    shape = _norm_args(x, groups, w, b, z, act, eps, center)
    dev = x.device
    _check("stats", stats, tuple(x.shape[:-1]) + (groups, 2), _F32, dev)
    _check("dy", dy, x.shape, x.dtype, dev)
    if not x.is_cuda:
        _require_cuda(x)
    workspace = _scratch("workspace", workspace, lib.gdn_norm_bwd_workspace_bytes(ctypes.byref(shape)), dev)
    like = lambda t, of: None if t is None else _empty_like(of)  # noqa: E731
    out = {"dx": _empty_like(dy), "dw": like(w, w), "db": like(b, b), "dz": like(z, dy)}
    rc = lib.gdn_norm_bwd(_byref(shape), x.data_ptr(), _at(w), _at(b), _at(z), stats.data_ptr(), dy.data_ptr(), _at(out["dx"]), _at(out["dw"]),
         _at(out["db"]), _at(out["dz"]), _at(workspace), _size(workspace), _stream_of(dev))
    if rc:
        _raise("gdn_norm_bwd", rc)
    return out


# ---------------------------------------------------------------------------------- projection
def _linear_args(x, W, bias, res, act):
    dev, dt = x.device, x.dtype
    lead, K = tuple(x.shape[:-1]), x.shape[-1]
    N = W.shape[0]
    M = x.numel() // max(K, 1)
    if x.numel() > INT_MAX or W.numel() > INT_MAX:
        _int_sizes("gdn_linear", M, N, K)
    ldx, ldw = _rows("x", x, lead + (K,), dt, dev), _rows("W", W, (N, K), dt, dev)
    if bias is not None:
        _check("bias", bias, (N,), dt, dev)
    ldres = 0 if res is None else _rows("res", res, lead + (N,), dt, dev)
    return GdnLinearShape(M, N, K, _act(act), _type(x), ldx, ldw, ldres), lead + (N,)


def gdn_linear_fwd_workspace_bytes(shape: GdnLinearShape) -> int:
    return _library().gdn_linear_fwd_workspace_bytes(ctypes.byref(shape))


def gdn_linear_bwd_workspace_bytes(shape: GdnLinearShape) -> int:
    return _library().gdn_linear_bwd_workspace_bytes(ctypes.byref(shape))


def gdn_linear_fwd(x, W, bias=None, res=None, *, act="none", y=None, pre=None, want_pre=False, workspace=None, stream=None):
    """y, pre = gdn_linear_fwd(x, W[, bias, res]) on CUDA tensors (see include/gdn.h):
    y = act(x W^T + bias) + res for x [..., K] and W [N, K]. pre (want_pre=True) is the
    pre-activation, which gdn_linear_bwd needs where act is not "none"."""
    if stream is not None:
        return _under(stream, gdn_linear_fwd, locals())
    lib = _library()
    shape, out_shape = _linear_args(x, W, bias, res, act)
    dev, dt = x.device, x.dtype
    if y is not None:
        _check("y", y, out_shape, dt, dev)
    if pre is not None:
        _check("pre", pre, out_shape, dt, dev)
    if not x.is_cuda:
        _require_cuda(x)
    if y is None:
        y = _empty(out_shape, dtype=dt, device=dev)
    if pre is None and want_pre:
        pre = _empty(out_shape, dtype=dt, device=dev)
    workspace = _scratch("workspace", workspace, lib.gdn_linear_fwd_workspace_bytes(ctypes.byref(shape)), dev)
    rc = lib.gdn_linear_fwd(_byref(shape), x.data_ptr(), W.data_ptr(), _at(bias), _at(res), _at(y), _at(pre), _at(workspace),
         _size(workspace), _stream_of(dev))
    if rc:
        _raise("gdn_linear_fwd", rc)
    return y, pre


def gdn_linear_bwd(x, W, dy, pre=None, *, act="none", want_dx=True, want_dW=True, want_dbias=True, workspace=None,
                   stream=None):
    """dict(dx, dW, dbias) = gdn_linear_bwd(x, W, dy[, pre]) for the inputs of gdn_linear_fwd (the
    gradient of res is dy itself). An entry is None with its want_... False."""
    if stream is not None:
        return _under(stream, gdn_linear_bwd, locals())
    lib = _library()
    shape, out_shape = _linear_args(x, W, None, None, act)
    dev, dt = x.device, x.dtype
    _check("dy", dy, out_shape, dt, dev)
    if pre is not None:
        _check("pre", pre, out_shape, dt, dev)
    if pre is None and shape.act != GDN_ACT_NONE:
        raise ValueError("pre is needed: the pre-activation of gdn_linear_fwd (want_pre=True)")
    if not x.is_cuda:
        _require_cuda(x)
    workspace = _scratch("workspace", workspace, lib.gdn_linear_bwd_workspace_bytes(ctypes.byref(shape)), dev)
    out = {"dx": _new_like(x) if want_dx else None,
           "dW": _new_like(W) if want_dW else None,
           "dbias": _empty((W.shape[0],), dtype=dt, device=dev) if want_dbias else None}
    rc = lib.gdn_linear_bwd(_byref(shape), x.data_ptr(), W.data_ptr(), _at(pre), dy.data_ptr(), _at(out["dx"]), _at(out["dW"]), _at(out["dbias"]),
         _at(workspace), _size(workspace), _stream_of(dev))
    if rc:
        _raise("gdn_linear_bwd", rc)
    return out


# ------------------------------------------------------------ linear attention with a decay
def _linattn_args(q, k, v, g, S0, lens):
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[-2:]
    dev, dt = q.device, q.dtype
    if q.numel() > INT_MAX or v.numel() > INT_MAX:
        _int_sizes("gdn_linattn", B, T, Hk, Hv, Dk, Dv)
    ldq, ldk = _rows("q", q, (B, T, Hk, Dk), dt, dev, 2), _rows("k", k, (B, T, Hk, Dk), dt, dev, 2)
    ldv = _rows("v", v, (B, T, Hv, Dv), dt, dev, 2)
    _check("g", g, (Hv,), _F32, dev)
    if S0 is not None:
        _check("S0", S0, (B, Hv, Dv, Dk), _F32, dev)
    if lens is not None:
        _check("lens", lens, (B,), _I32, dev)
    return _linattn_shape(B, T, Hk, Hv, Dk, Dv, _type(q), ldq, ldk, ldv), B, T, Hv, Dk, Dv


def gdn_linattn_fwd_workspace_bytes(shape: GdnLinattnShape) -> int:
    return _library().gdn_linattn_fwd_workspace_bytes(ctypes.byref(shape))


def gdn_linattn_bwd_workspace_bytes(shape: GdnLinattnShape) -> int:
    return _library().gdn_linattn_bwd_workspace_bytes(ctypes.byref(shape))


def gdn_linattn_fwd(q, k, v, g, S0=None, lens=None, *, y=None, S_T=None, workspace=None, want_S_T=True, stream=None):
    """y, S_T = gdn_linattn_fwd(q, k, v, g[, S0, lens]) on CUDA tensors (see include/gdn.h): linear
    attention of q, k [B, T, Hk, Dk] and v [B, T, Hv, Dv] whose state [B, Hv, Dv, Dk] decays by g [Hv] at
    every step. With T = 1, S_T may be S0: the state updated in place."""
    if stream is not None:
        return _under(stream, gdn_linattn_fwd, locals())
    lib = _library()
    shape, B, T, Hv, Dk, Dv = _linattn_args(q, k, v, g, S0, lens)
    dev, dt = q.device, q.dtype
    if y is not None:
        _check("y", y, (B, T, Hv, Dv), dt, dev)
    if S_T is not None:
        _check("S_T", S_T, (B, Hv, Dv, Dk), _F32, dev)
    if not q.is_cuda:
        _require_cuda(q)
    if y is None:
        y = _new_like(v)
    if S_T is None and want_S_T:
        S_T = _empty((B, Hv, Dv, Dk), dtype=_F32, device=dev) if S0 is None else _empty_like(S0)
    if workspace is not None or T > 1:                 # a single step needs none
        workspace = _scratch("workspace", workspace, lib.gdn_linattn_fwd_workspace_bytes(_byref(shape)), dev)
    rc = lib.gdn_linattn_fwd(_byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _at(S0), _at(lens), _at(y), _at(S_T),
                             _at(workspace), _size(workspace), _stream_of(dev))
    if rc:
        _raise("gdn_linattn_fwd", rc)
    return y, S_T


def gdn_linattn_bwd(q, k, v, g, dy, S0=None, lens=None, dS_T=None, *, workspace=None, want_dS0=True, stream=None):
    """dict(dq, dk, dv, dS0) = gdn_linattn_bwd(q, k, v, g, dy, ...) for the inputs of gdn_linattn_fwd.
    dS0 is None with want_dS0=False."""
    if stream is not None:
        return _under(stream, gdn_linattn_bwd, locals())
    lib = _library()
    shape, B, T, Hv, Dk, Dv = _linattn_args(q, k, v, g, S0, lens)
    dev, dt = q.device, q.dtype
    _check("dy", dy, (B, T, Hv, Dv), dt, dev)
    if dS_T is not None:
        _check("dS_T", dS_T, (B, Hv, Dv, Dk), _F32, dev)
    if not q.is_cuda:
        _require_cuda(q)
    workspace = _scratch("workspace", workspace, lib.gdn_linattn_bwd_workspace_bytes(_byref(shape)), dev)
    out = {"dq": _new_like(q), "dk": _new_like(k), "dv": _empty_like(dy),
           "dS0": _empty((B, Hv, Dv, Dk), dtype=_F32, device=dev) if want_dS0 else None}
    rc = lib.gdn_linattn_bwd(_byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _at(S0), _at(lens), dy.data_ptr(), _at(dS_T),
         _at(out["dq"]), _at(out["dk"]), _at(out["dv"]), _at(out["dS0"]), _at(workspace), _size(workspace), _stream_of(dev))
    if rc:
        _raise("gdn_linattn_bwd", rc)
    return out


# ------------------------------------------------------------------------ norms around a block
def _resnorm_args(x, h, z, scale, w_post, w_pre, post, pre, act, eps):
    dev, dt, size = x.device, x.dtype, x.shape
    D, n = size[-1], x.numel()
    rows, gate_rows = n // max(D, 1), 1
    if n > INT_MAX:
        _int_sizes("gdn_resnorm", rows, D)
    ldx, ldh, ldz = _rows("x", x, size, dt, dev), _rows("h", h, size, dt, dev), 0
    if z is not None:
        lead = z.dim() - 1
        if lead < 0 or lead >= x.dim() or z.shape[-1] != D or z.shape[:lead] != size[:lead]:
            raise ValueError(f"z has shape {tuple(z.shape)}, expected {tuple(size)} or its last dimension behind some of its first ones")
        gate_rows = rows // max(z.numel() // max(D, 1), 1)
        ldz = _rows("z", z, z.shape, dt, dev)
    if scale is not None:
        _check("scale", scale, (D,), _F32, dev)
    if w_post is not None:
        if not post:
            raise ValueError("w_post is given, but its norm is off")
        _check("w_post", w_post, (D,), _F32, dev)
    if w_pre is not None:
        if not pre:
            raise ValueError("w_pre is given, but its norm is off")
        _check("w_pre", w_pre, (D,), _F32, dev)
    return _resnorm_shape(rows, D, gate_rows, _act(act), 1 if post else 0, 1 if pre else 0, _type(x), float(eps), ldx, ldh, ldz)


def gdn_resnorm_fwd(x, h, z=None, scale=None, w_post=None, w_pre=None, *, post=True, pre=True, act="none", eps=1e-5, r=None, y=None,
                    stats=None, want_stats=True, stream=None):
    """r, y, stats = gdn_resnorm_fwd(x, h[, z, scale, w_post, w_pre]) on CUDA tensors (see include/gdn.h):
    r = x + scale act(z) norm(h) w_post, y = norm(r) w_pre, root mean square norms over the last
    dimension. z has x's shape, or some of its first dimensions and the last ([B, D] for x [B, T, D]: a row
    for each sequence). post=False: h is added as it is; pre=False: y is None. r may be x (packed): the
    stream updated in place. stats [..., 2] is what gdn_resnorm_bwd needs."""
    if stream is not None:
        return _under(stream, gdn_resnorm_fwd, locals())
    lib = _library()
    shape = _resnorm_args(x, h, z, scale, w_post, w_pre, post, pre, act, eps)
    dev, dt = x.device, x.dtype
    if r is not None:
        _check("r", r, x.shape, dt, dev)
    if y is not None:
        if not pre:
            raise ValueError("y is given, but its norm is off")
        _check("y", y, x.shape, dt, dev)
    if stats is not None:
        _check("stats", stats, x.shape[:-1] + (2,), _F32, dev)
    if not x.is_cuda:
        _require_cuda(x)
    if r is None:
        r = _new_like(x)
    if y is None and pre:
        y = _new_like(x)
    if stats is None and want_stats:
        stats = _empty(x.shape[:-1] + (2,), dtype=_F32, device=dev)
    rc = lib.gdn_resnorm_fwd(_byref(shape), x.data_ptr(), h.data_ptr(), _at(z), _at(scale), _at(w_post), _at(w_pre), r.data_ptr(), _at(y),
                             _at(stats), _stream_of(dev))
    if rc:
        _raise("gdn_resnorm_fwd", rc)
    return r, y, stats


def gdn_resnorm_bwd_workspace_bytes(shape: GdnResnormShape) -> int:
    return _library().gdn_resnorm_bwd_workspace_bytes(ctypes.byref(shape))


def gdn_resnorm_bwd(x, h, stats, dy=None, dr=None, z=None, scale=None, w_post=None, w_pre=None, *, post=True, pre=True, act="none", eps=1e-5,
                    workspace=None, stream=None):
    """dict(dx, dh, dz, dscale, dw_post, dw_pre) = gdn_resnorm_bwd(x, h, stats, dy, dr[, z, scale, w_post,
    w_pre]) for the inputs and stats of gdn_resnorm_fwd and the gradients of y (None with pre=False) and r
    (None: zeros). dz, dscale, dw_post and dw_pre (float32) are None where their input was."""
    if stream is not None:
        return _under(stream, gdn_resnorm_bwd, locals())
    lib = _library()
    shape = _resnorm_args(x, h, z, scale, w_post, w_pre, post, pre, act, eps)
    dev, dt = x.device, x.dtype
    _check("stats", stats, x.shape[:-1] + (2,), _F32, dev)
    if (dy is None) == bool(pre):
        raise ValueError("dy is needed: the gradient of y" if pre else "dy is given, but its norm is off")
    if dy is not None:
        _check("dy", dy, x.shape, dt, dev)
    if dr is not None:
        _check("dr", dr, x.shape, dt, dev)
    elif not pre:
        raise ValueError("dr is needed: the gradient of r")
    if not x.is_cuda:
        _require_cuda(x)
    workspace = _scratch("workspace", workspace, lib.gdn_resnorm_bwd_workspace_bytes(_byref(shape)), dev)
    vec = lambda t: None if t is None else _empty_like(t)  # noqa: E731
    out = {"dx": _new_like(x), "dh": _new_like(h), "dz": None if z is None else _new_like(z), "dscale": vec(scale),
           "dw_post": vec(w_post), "dw_pre": vec(w_pre)}
    rc = lib.gdn_resnorm_bwd(_byref(shape), x.data_ptr(), h.data_ptr(), _at(z), _at(scale), _at(w_post), _at(w_pre), stats.data_ptr(), _at(dy),
         _at(dr), _at(out["dx"]), _at(out["dh"]), _at(out["dz"]), _at(out["dscale"]), _at(out["dw_post"]), _at(out["dw_pre"]),
         _at(workspace), _size(workspace), _stream_of(dev))
    if rc:
        _raise("gdn_resnorm_bwd", rc)
    return out

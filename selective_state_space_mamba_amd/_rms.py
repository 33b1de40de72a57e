"""Binding of the root-mean-square norm with the residual's addition
(mamba_rms_norm_*, include/mamba_scan.h): x [..., D] float32 or bfloat16,
s = x + residual as stored, out = s·rstd·weight, rounded to x's type or to
8 bits with a scale a row."""
from __future__ import annotations

import ctypes
import functools

from . import _binding as _b
from ._call import check_f32, check_like, done, launch_stream, ptr, query, use_workspace


class RmsDims(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("dim", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("residual_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


def declare(lib):
    vp, dims = ctypes.c_void_p, ctypes.POINTER(RmsDims)
    fn = lib.mamba_rms_norm_bwd_workspace_bytes
    fn.restype, fn.argtypes = ctypes.c_size_t, [dims]
    for name in ("fwd", "q8"):
        fn = getattr(lib, "mamba_rms_norm_" + name)
        fn.restype, fn.argtypes = ctypes.c_int, [vp] * 3 + [dims] + [vp] * 4
    lib.mamba_rms_norm_bwd.restype = ctypes.c_int
    lib.mamba_rms_norm_bwd.argtypes = [vp] * 5 + [dims] + [vp] * 4


def make_rms_dims(rows, dim, dtype, *, residual_dtype=None, eps=1e-5, workspace=None, workspace_bytes=0) -> RmsDims:
    return RmsDims(int(rows), int(dim), int(dtype), int(dtype if residual_dtype is None else residual_dtype), float(eps),
                   _b._ptr(workspace), int(workspace_bytes))


def rms_norm_bwd_workspace_bytes(dims: RmsDims) -> int:
    return query("mamba_rms_norm_bwd_workspace_bytes", dims)


@functools.lru_cache(maxsize=512)
def _bwd_bytes(rows, D, dt, rt):
    """A pure function of the sizes and types."""
    return rms_norm_bwd_workspace_bytes(make_rms_dims(rows, D, dt, residual_dtype=rt))


@functools.lru_cache(maxsize=512)
def _bare_dims(rows, D, dt, rt, eps):
    """A reference to the sizes of a forward, which only reads them."""
    return ctypes.byref(make_rms_dims(rows, D, dt, residual_dtype=rt, eps=eps))


def _check_inputs(x, weight):
    shape = x.shape
    if len(shape) < 1:
        raise ValueError("x must be [..., D], got a scalar")
    dt = _b._dtype_code(x)
    if not x.is_contiguous():
        check_like(x, shape, ("x", x))  # raises with the reason
    D = shape[-1]
    if weight is not None:
        check_f32(x, (D,), ("weight", weight))
    return x.numel() // D if D else 0, D, shape, dt


def _stream_code(x, dt, shape, name, t):
    """The type's code of the residual stream t: x's type, or float32."""
    rt = _b._dtype_code(t)
    if rt != dt and rt != _b.DTYPE_F32:
        raise TypeError("%s must be float32 or of x's type, got %s for %s" % (name, t.dtype, x.dtype))
    if not (t.shape == shape and t.is_contiguous() and t.get_device() == x.get_device()):
        _b._check(t, name, shape, t.dtype, x.device)  # raises with the reason
    return rt


def _fwd(x, weight, residual, eps, added):
    """What both forward forms check: (shape, dims, added)."""
    import torch
    rows, D, shape, dt = _check_inputs(x, weight)
    if residual is None:
        if added is not None:
            raise ValueError("added is what x and residual add up to; there is no residual")
        return shape, _bare_dims(rows, D, dt, dt, float(eps)), None
    rt = _stream_code(x, dt, shape, "residual", residual)
    if added is None:
        added = torch.empty_like(residual)
    else:
        check_like(residual, shape, ("added", added))
    return shape, _bare_dims(rows, D, dt, rt, float(eps)), added


def rms_norm_fwd(x, weight=None, residual=None, *, eps=1e-5, out=None, added=None, rstd=None, stream=None):
    """mamba_rms_norm_fwd on torch tensors: x [..., D], weight [D] float32,
    residual [..., D] of x's type or float32.  Returns (out, added, rstd): added
    is x + residual in the residual's type (None without one; residual itself
    may be given for it), rstd [...] float32 what rms_norm_bwd takes.  out may
    be x itself."""
    import torch
    ts = None if stream is None else _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return rms_norm_fwd(x, weight, residual, eps=eps, out=out, added=added, rstd=rstd, stream=ts)
    shape, dims, added = _fwd(x, weight, residual, eps, added)
    raw = launch_stream(x, stream)
    if out is None:
        out = torch.empty_like(x)
    else:
        check_like(x, shape, ("out", out))
    if rstd is None:
        rstd = x.new_empty(shape[:-1], dtype=torch.float32)
    else:
        check_f32(x, shape[:-1], ("rstd", rstd))
    done(_b.load_library().mamba_rms_norm_fwd(x.data_ptr(), ptr(residual), ptr(weight), dims,
                                              out.data_ptr(), ptr(added), rstd.data_ptr(), raw), "mamba_rms_norm_fwd")
    return out, added, rstd


def rms_norm_q8(x, weight=None, residual=None, *, eps=1e-5, out=None, scale=None, added=None, stream=None):
    """mamba_rms_norm_q8 on torch tensors, arguments as for rms_norm_fwd.
    Returns (out [..., D] float8_e4m3fn, scale [...] float32, added): the
    normalised row is out·scale."""
    import torch
    ts = None if stream is None else _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return rms_norm_q8(x, weight, residual, eps=eps, out=out, scale=scale, added=added, stream=ts)
    shape, dims, added = _fwd(x, weight, residual, eps, added)
    raw = launch_stream(x, stream)
    if out is None:
        out = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    else:
        _b._check(out, "out", shape, torch.float8_e4m3fn, x.device)
    if scale is None:
        scale = x.new_empty(shape[:-1], dtype=torch.float32)
    else:
        check_f32(x, shape[:-1], ("scale", scale))
    done(_b.load_library().mamba_rms_norm_q8(x.data_ptr(), ptr(residual), ptr(weight), dims,
                                             out.data_ptr(), scale.data_ptr(), ptr(added), raw), "mamba_rms_norm_q8")
    return out, scale, added


def rms_norm_bwd(s, weight=None, *, dout, rstd, dadded=None, want_dweight=True, workspace=None, stream=None):
    """mamba_rms_norm_bwd on torch tensors: s is what rms_norm_fwd normalised
    (added, or x without a residual), rstd what it returned, dout [..., D] the
    gradient of out, dadded (of s's type) that of added.  Returns a dict with
    dx (of dout's type), dresidual (of s's type: dx itself where the types are
    the same) and dweight (None without a weight, or unless wanted)."""
    import torch
    ts = None if stream is None else _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return rms_norm_bwd(s, weight, dout=dout, rstd=rstd, dadded=dadded, want_dweight=want_dweight,
                                workspace=workspace, stream=ts)
    rows, D, shape, dt = _check_inputs(dout, weight)
    rt = _stream_code(dout, dt, shape, "s", s)
    check_like(s, shape, ("dadded", dadded))
    check_f32(dout, shape[:-1], ("rstd", rstd))
    raw = launch_stream(dout, stream)
    dims = make_rms_dims(rows, D, dt, residual_dtype=rt)
    want_dweight = want_dweight and weight is not None
    need = _bwd_bytes(rows, D, dt, rt) if want_dweight else 0
    workspace = use_workspace(dims, need, workspace, dout)
    dx = torch.empty_like(dout)
    dresidual = dx if rt == dt else torch.empty_like(s)
    dweight = torch.empty_like(weight) if want_dweight else None
    done(_b.load_library().mamba_rms_norm_bwd(s.data_ptr(), ptr(weight), rstd.data_ptr(), dout.data_ptr(), ptr(dadded),
                                              ctypes.byref(dims), dx.data_ptr(),
                                              None if dresidual is dx else dresidual.data_ptr(), ptr(dweight), raw),
         "mamba_rms_norm_bwd")
    return dict(dx=dx, dresidual=dresidual, dweight=dweight)

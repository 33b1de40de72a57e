"""Bindings of the products with quantised weights (mamba_linear_q8 and
mamba_linear_q4, include/mamba_scan.h): rows and weights in e4m3 with a scale
for each row of either, and weights of 4 bits with a scale for each group."""
from __future__ import annotations

import ctypes
import functools

from . import _binding as _b
from ._call import check_f32, check_like, done, launch_stream, ptr, query, use_workspace
from ._linear import LinearDims, make_linear_dims
from ._norm import ACT_NONE


class Q4Dims(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("in_dim", ctypes.c_int64), ("out_dim", ctypes.c_int64), ("group", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("scale_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
    ]


def declare(lib):
    vp = ctypes.c_void_p
    lib.mamba_linear_q8_workspace_bytes.restype = ctypes.c_size_t
    lib.mamba_linear_q8_workspace_bytes.argtypes = [ctypes.POINTER(LinearDims)]
    lib.mamba_linear_q8.restype = ctypes.c_int
    lib.mamba_linear_q8.argtypes = [vp] * 6 + [ctypes.POINTER(LinearDims)] + [vp] * 2
    lib.mamba_linear_q4.restype = ctypes.c_int
    lib.mamba_linear_q4.argtypes = [vp] * 6 + [ctypes.POINTER(Q4Dims)] + [vp] * 2


def make_q4_dims(rows, in_dim, out_dim, group, dtype, *, scale_dtype=None, act=ACT_NONE) -> Q4Dims:
    return Q4Dims(int(rows), int(in_dim), int(out_dim), int(group), int(dtype),
                  int(dtype if scale_dtype is None else scale_dtype), int(act))


def linear_q8_workspace_bytes(dims: LinearDims) -> int:
    return query("mamba_linear_q8_workspace_bytes", dims)


@functools.lru_cache(maxsize=512)
def _q8_bytes(M, K, N):
    """A pure function of the sizes."""
    return linear_q8_workspace_bytes(make_linear_dims(M, K, N, _b.DTYPE_BF16))


@functools.lru_cache(maxsize=512)
def _bare_q8_dims(M, K, N, dt, act):
    """A reference to the sizes of a call without workspace, which only reads them."""
    return ctypes.byref(make_linear_dims(M, K, N, dt, act=act))


@functools.lru_cache(maxsize=512)
def _q4_dims(*sizes):
    return ctypes.byref(Q4Dims(*sizes))


def _out_shape(xs, N):
    return (xs[0], N) if len(xs) == 2 else tuple(xs[:-1]) + (N,)


def linear_q8(x, x_scale, weight, w_scale, bias=None, residual=None, *, act=ACT_NONE, dtype=None, out=None,
              workspace=None, stream=None):
    """mamba_linear_q8 on torch tensors: x [..., K] and weight [N][K]
    float8_e4m3fn, x_scale [...] and w_scale [N] float32 (a row is x·x_scale),
    bias [N] float32, residual and out [..., N] float32 or bfloat16 (out may be
    residual).  Returns out; its type is out's, residual's or dtype, bfloat16
    where none is given.  Products are added in float32 where it is float32, and
    for few rows; otherwise each eight neighbouring ones lose what lies below
    2^-13 of the largest (mamba_scan.h)."""
    import torch
    ts = None if stream is None else _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return linear_q8(x, x_scale, weight, w_scale, bias, residual, act=act, dtype=dtype, out=out,
                             workspace=workspace, stream=ts)
    xs, wsh = x.shape, weight.shape
    if len(wsh) != 2 or len(xs) < 1 or xs[-1] != wsh[1]:
        raise ValueError("x must be [..., K] and weight [N][K], got %s and %s" % (tuple(xs), tuple(wsh)))
    e4m3, f32, dev = torch.float8_e4m3fn, torch.float32, x.get_device()
    N, K = wsh
    # (written out: a step is a few microseconds)
    if not (x.dtype is e4m3 and weight.dtype is e4m3 and x.is_contiguous() and weight.is_contiguous()
            and x_scale.shape == xs[:-1] and x_scale.dtype is f32 and x_scale.is_contiguous()
            and w_scale.shape == wsh[:1] and w_scale.dtype is f32 and w_scale.is_contiguous()
            and weight.get_device() == dev and x_scale.get_device() == dev and w_scale.get_device() == dev):
        if x.dtype is not e4m3:
            raise TypeError("x must be float8_e4m3fn, got %s" % x.dtype)
        check_like(x, xs, ("x", x))
        check_like(x, wsh, ("weight", weight))
        check_f32(x, xs[:-1], ("x_scale", x_scale))
        check_f32(x, (N,), ("w_scale", w_scale))
    raw = launch_stream(x, stream)
    M = x.numel() // K if K else 0
    if bias is not None:
        check_f32(x, (N,), ("bias", bias))
    shape = _out_shape(xs, N)
    given = residual if out is None else out
    if given is not None:
        dt = _b._dtype_code(given)
        if dtype is not None and given.dtype is not dtype:
            raise TypeError("out and residual must be %s, got %s" % (dtype, given.dtype))
        for name, t in (("out", out), ("residual", residual)):
            _b._check(t, name, shape, given.dtype, x.device)
    if out is None:
        out = x.new_empty(shape, dtype=torch.bfloat16 if dtype is None else dtype) if given is None else torch.empty_like(given)
        dt = _b._dtype_code(out)
    need, act = _q8_bytes(M, K, N), int(act)  # (a tensor would be looked up by its identity)
    if need == 0 and workspace is None:
        dims = _bare_q8_dims(M, K, N, dt, act)
    else:
        held = make_linear_dims(M, K, N, dt, act=act)
        workspace = use_workspace(held, need, workspace, x)
        dims = ctypes.byref(held)
    done(_b.load_library().mamba_linear_q8(x.data_ptr(), x_scale.data_ptr(), weight.data_ptr(), w_scale.data_ptr(),
                                           ptr(bias), ptr(residual), dims, out.data_ptr(), raw),
         "mamba_linear_q8")
    return out


def linear_q4(x, weight, scale, zero=None, bias=None, residual=None, *, group=128, act=ACT_NONE, out=None, stream=None):
    """mamba_linear_q4 on torch tensors: x [..., K] float32 or bfloat16, weight
    [N][K/2] uint8 (two weights a byte, the even element's in the low four bits),
    scale [N][ceil(K/group)] float32 or bfloat16, zero of the same shape uint8
    (any byte; None: 8), bias [N] float32, residual and out [..., N] of x's type (out may
    be residual).  A weight stands for (q - zero)·scale.  Returns out."""
    import torch
    ts = None if stream is None else _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return linear_q4(x, weight, scale, zero, bias, residual, group=group, act=act, out=out, stream=ts)
    xs, wsh = x.shape, weight.shape
    if len(wsh) != 2 or len(xs) < 1 or xs[-1] != 2 * wsh[1]:
        raise ValueError("x must be [..., K] and weight [N][K/2], got %s and %s" % (tuple(xs), tuple(wsh)))
    dt = _b._dtype_code(x)
    if not x.is_contiguous():
        check_like(x, xs, ("x", x))  # raises with the reason
    raw = launch_stream(x, stream)
    N, K = wsh[0], xs[-1]
    group = int(group)
    if group <= 0:
        raise ValueError("group must be positive, got %d" % group)
    table = (N, -(-K // group))
    _b._check(weight, "weight", wsh, torch.uint8, x.device)
    scale_dt = _b._dtype_code(scale)
    _b._check(scale, "scale", table, scale.dtype, x.device)
    _b._check(zero, "zero", table, torch.uint8, x.device)
    if bias is not None:
        check_f32(x, (N,), ("bias", bias))
    shape = _out_shape(xs, N)
    if residual is not None or out is not None:
        check_like(x, shape, ("residual", residual), ("out", out))
    if out is None:
        out = x.new_empty(shape) if residual is None else torch.empty_like(residual)
    dims = _q4_dims(x.numel() // K if K else 0, K, N, group, dt, scale_dt, int(act))
    done(_b.load_library().mamba_linear_q4(x.data_ptr(), weight.data_ptr(), scale.data_ptr(), ptr(zero), ptr(bias),
                                           ptr(residual), dims, out.data_ptr(), raw), "mamba_linear_q4")
    return out

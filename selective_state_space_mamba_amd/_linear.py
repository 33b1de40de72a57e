"""Binding of the matrix product with bias, activation and residual
(mamba_linear_*, include/mamba_scan.h):
out = act(x·weightᵀ + bias) + residual for x [..., K] and weight [N][K]."""
from __future__ import annotations

import ctypes

from . import _binding as _b
from ._glr import _query, _workspace
from ._norm import ACT_NONE


class LinearDims(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("in_dim", ctypes.c_int64), ("out_dim", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("act", ctypes.c_int32),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


def declare(lib):
    vp, dims = ctypes.c_void_p, ctypes.POINTER(LinearDims)
    for name in ("fwd_workspace_bytes", "bwd_workspace_bytes"):
        fn = getattr(lib, "mamba_linear_" + name)
        fn.restype, fn.argtypes = ctypes.c_size_t, [dims]
    lib.mamba_linear_fwd.restype = ctypes.c_int
    lib.mamba_linear_fwd.argtypes = [vp] * 4 + [dims] + [vp] * 3
    lib.mamba_linear_bwd.restype = ctypes.c_int
    lib.mamba_linear_bwd.argtypes = [vp] * 4 + [dims] + [vp] * 4


def make_linear_dims(rows, in_dim, out_dim, dtype, *, act=ACT_NONE, workspace=None, workspace_bytes=0) -> LinearDims:
    return LinearDims(int(rows), int(in_dim), int(out_dim), int(dtype), int(act), _b._ptr(workspace),
                      int(workspace_bytes))


def linear_fwd_workspace_bytes(dims: LinearDims) -> int:
    return _query("mamba_linear_fwd_workspace_bytes", dims)


def linear_bwd_workspace_bytes(dims: LinearDims) -> int:
    return _query("mamba_linear_bwd_workspace_bytes", dims)


def _check_inputs(x, weight):
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x must be [..., K] and weight [N][K], got %s and %s" % (tuple(x.shape), tuple(weight.shape)))
    N, K = weight.shape
    _b._check(x, "x", tuple(x.shape), x.dtype, x.device)
    _b._check(weight, "weight", (N, K), x.dtype, x.device)
    return x.numel() // K if K else 0, K, N, tuple(x.shape[:-1]) + (N,), _b._dtype_code(x), x.device


def linear_fwd(x, weight, bias=None, residual=None, *, act=ACT_NONE, out=None, pre=None, want_pre=False,
               workspace=None, stream=None):
    """mamba_linear_fwd on torch tensors: x [..., K], weight [N][K], bias [N]
    float32, residual and out [..., N] (out may be residual).  Returns (out,
    pre); pre is the product before the activation, [..., N] float32, which
    linear_bwd takes (None unless want_pre or a buffer for it is given)."""
    import torch
    ts = _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return linear_fwd(x, weight, bias, residual, act=act, out=out, pre=pre, want_pre=want_pre,
                              workspace=workspace, stream=ts)
    lib = _b.load_library()
    M, K, N, shape, dt, dev = _check_inputs(x, weight)
    _b._check(bias, "bias", (N,), torch.float32, dev)
    _b._check(residual, "residual", shape, x.dtype, dev)
    dims = make_linear_dims(M, K, N, dt, act=act)
    workspace = _workspace(dims, linear_fwd_workspace_bytes(dims), workspace, dev)
    out = torch.empty(shape, dtype=x.dtype, device=dev) if out is None else out
    if pre is None and want_pre:
        pre = torch.empty(shape, dtype=torch.float32, device=dev)
    _b._check(out, "out", shape, x.dtype, dev)
    _b._check(pre, "pre", shape, torch.float32, dev)
    rc = lib.mamba_linear_fwd(_b._ptr(x), _b._ptr(weight), _b._ptr(bias), _b._ptr(residual), ctypes.byref(dims),
                              _b._ptr(out), _b._ptr(pre), _b._stream(stream))
    if rc != _b.MAMBA_OK:
        raise _b.MambaError(rc, "mamba_linear_fwd")
    return out, pre


def linear_bwd(x, weight, *, dout, pre=None, act=ACT_NONE, want_dx=True, want_dweight=True, want_dbias=True,
               workspace=None, stream=None):
    """mamba_linear_bwd on torch tensors, with the pre that linear_fwd returned
    (needed with an activation).  Returns a dict with dx, dweight (None unless
    wanted) and dbias [N] float32; the residual's gradient is dout."""
    import torch
    ts = _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return linear_bwd(x, weight, dout=dout, pre=pre, act=act, want_dx=want_dx, want_dweight=want_dweight,
                              want_dbias=want_dbias, workspace=workspace, stream=ts)
    lib = _b.load_library()
    M, K, N, shape, dt, dev = _check_inputs(x, weight)
    _b._check(dout, "dout", shape, x.dtype, dev)
    _b._check(pre, "pre", shape, torch.float32, dev)
    dims = make_linear_dims(M, K, N, dt, act=act)
    workspace = _workspace(dims, linear_bwd_workspace_bytes(dims), workspace, dev)
    g = dict(dx=torch.empty_like(x) if want_dx else None, dweight=torch.empty_like(weight) if want_dweight else None,
             dbias=torch.empty(N, dtype=torch.float32, device=dev) if want_dbias else None)
    rc = lib.mamba_linear_bwd(_b._ptr(x), _b._ptr(weight), _b._ptr(pre), _b._ptr(dout), ctypes.byref(dims),
                              _b._ptr(g["dx"]), _b._ptr(g["dweight"]), _b._ptr(g["dbias"]), _b._stream(stream))
    if rc != _b.MAMBA_OK:
        raise _b.MambaError(rc, "mamba_linear_bwd")
    return g

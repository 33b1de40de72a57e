"""Binding of the matrix product with bias, activation and residual
(mamba_linear_*, include/mamba_scan.h):
out = act(x·weightᵀ + bias) + residual for x [..., K] and weight [N][K]."""
from __future__ import annotations

import ctypes
import functools

from . import _binding as _b
from ._call import check_f32, check_like, done, launch_stream, ptr, query, use_workspace
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
    lib.mamba_linear_plan.restype = ctypes.c_int
    lib.mamba_linear_plan.argtypes = [dims, ctypes.c_int] + [ctypes.POINTER(ctypes.c_int32)] * 3
    lib.mamba_linear_fwd.restype = ctypes.c_int
    lib.mamba_linear_fwd.argtypes = [vp] * 4 + [dims] + [vp] * 3
    lib.mamba_linear_bwd.restype = ctypes.c_int
    lib.mamba_linear_bwd.argtypes = [vp] * 4 + [dims] + [vp] * 4


def make_linear_dims(rows, in_dim, out_dim, dtype, *, act=ACT_NONE, workspace=None, workspace_bytes=0) -> LinearDims:
    return LinearDims(int(rows), int(in_dim), int(out_dim), int(dtype), int(act), _b._ptr(workspace),
                      int(workspace_bytes))


def linear_fwd_workspace_bytes(dims: LinearDims) -> int:
    return query("mamba_linear_fwd_workspace_bytes", dims)


def linear_bwd_workspace_bytes(dims: LinearDims) -> int:
    return query("mamba_linear_bwd_workspace_bytes", dims)


def linear_plan(dims: LinearDims, product: int):
    """mamba_linear_plan: (tile rows, tile columns, shares of the contraction) of product 0 (forward), 1 (dx) or 2 (dweight)."""
    out = [ctypes.c_int32() for _ in range(3)]
    done(_b.load_library().mamba_linear_plan(ctypes.byref(dims), int(product), *(ctypes.byref(v) for v in out)),
         "mamba_linear_plan")
    return tuple(v.value for v in out)


@functools.lru_cache(maxsize=512)
def _sizes(M, K, N, dt, act):
    """(forward, backward) workspace: pure functions of the sizes."""
    d = make_linear_dims(M, K, N, dt, act=act)
    return linear_fwd_workspace_bytes(d), linear_bwd_workspace_bytes(d)


def _check_inputs(x, weight):
    xs, ws = x.shape, weight.shape
    if len(ws) != 2 or len(xs) < 1 or xs[-1] != ws[1]:
        raise ValueError("x must be [..., K] and weight [N][K], got %s and %s" % (tuple(xs), tuple(ws)))
    dt = _b._dtype_code(x)
    check_like(x, xs, ("x", x))
    check_like(x, ws, ("weight", weight))
    N, K = ws
    return x.numel() // K if K else 0, K, N, xs[:-1] + ws[:1], dt


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
    M, K, N, shape, dt = _check_inputs(x, weight)
    raw = launch_stream(x, stream)
    if bias is not None:
        check_f32(x, (N,), ("bias", bias))
    check_like(x, shape, ("residual", residual), ("out", out))
    act = int(act)  # (a tensor would be looked up below by its identity)
    need, _ = _sizes(M, K, N, dt, act)
    dims = make_linear_dims(M, K, N, dt, act=act)
    workspace = use_workspace(dims, need, workspace, x)
    if out is None:
        out = x.new_empty(shape) if residual is None else torch.empty_like(residual)
    if pre is not None:
        check_f32(x, shape, ("pre", pre))
    elif want_pre:
        pre = torch.empty(shape, dtype=torch.float32, device=x.device)
    done(_b.load_library().mamba_linear_fwd(x.data_ptr(), weight.data_ptr(), ptr(bias), ptr(residual),
                                            ctypes.byref(dims), out.data_ptr(), ptr(pre), raw), "mamba_linear_fwd")
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
    M, K, N, shape, dt = _check_inputs(x, weight)
    raw = launch_stream(x, stream)
    check_like(x, shape, ("dout", dout))
    if pre is not None:
        check_f32(x, shape, ("pre", pre))
    act = int(act)
    _, need = _sizes(M, K, N, dt, act)
    dims = make_linear_dims(M, K, N, dt, act=act)
    workspace = use_workspace(dims, need, workspace, x)
    dx = torch.empty_like(x) if want_dx else None
    dweight = torch.empty_like(weight) if want_dweight else None
    dbias = torch.empty(N, dtype=torch.float32, device=x.device) if want_dbias else None
    done(_b.load_library().mamba_linear_bwd(x.data_ptr(), weight.data_ptr(), ptr(pre), dout.data_ptr(),
                                            ctypes.byref(dims), ptr(dx), ptr(dweight), ptr(dbias), raw),
         "mamba_linear_bwd")
    return dict(dx=dx, dweight=dweight, dbias=dbias)

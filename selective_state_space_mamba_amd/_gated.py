"""Binding of the gated pair of products (mamba_gated_linear_*,
include/mamba_scan.h): out = act(x·w_gateᵀ + b_gate)·(x·w_upᵀ + b_up) for x
[..., K] and weights [N][K]."""
from __future__ import annotations

import ctypes
import functools

from . import _binding as _b
from ._call import check_f32, check_like, done, launch_stream, ptr, query, use_workspace
from ._linear import LinearDims, _check_inputs, make_linear_dims
from ._norm import ACT_SILU


def declare(lib):
    vp, dims = ctypes.c_void_p, ctypes.POINTER(LinearDims)
    for name in ("fwd_workspace_bytes", "bwd_workspace_bytes"):
        fn = getattr(lib, "mamba_gated_linear_" + name)
        fn.restype, fn.argtypes = ctypes.c_size_t, [dims]
    lib.mamba_gated_linear_fwd.restype = ctypes.c_int
    lib.mamba_gated_linear_fwd.argtypes = [vp] * 5 + [dims] + [vp] * 3
    lib.mamba_gated_linear_bwd.restype = ctypes.c_int
    lib.mamba_gated_linear_bwd.argtypes = [vp] * 5 + [dims] + [vp] * 6


def gated_linear_fwd_workspace_bytes(dims: LinearDims) -> int:
    return query("mamba_gated_linear_fwd_workspace_bytes", dims)


def gated_linear_bwd_workspace_bytes(dims: LinearDims) -> int:
    return query("mamba_gated_linear_bwd_workspace_bytes", dims)


@functools.lru_cache(maxsize=512)
def _sizes(M, K, N, dt):
    """(forward, backward) workspace: pure functions of the sizes."""
    d = make_linear_dims(M, K, N, dt)
    return gated_linear_fwd_workspace_bytes(d), gated_linear_bwd_workspace_bytes(d)


@functools.lru_cache(maxsize=512)
def _bare_dims(M, K, N, dt, act):
    """A reference to the sizes of a call without workspace, which only reads them."""
    return ctypes.byref(make_linear_dims(M, K, N, dt, act=act))


def _check_all(x, w_gate, w_up):
    """(M, K, N, the output's shape, the type's code).  The checks are written out: a step is a few microseconds."""
    xs, ws, dtype, dev = x.shape, w_gate.shape, x.dtype, x.get_device()
    if not (len(ws) == 2 and len(xs) >= 1 and xs[-1] == ws[1] and w_up.shape == ws and w_gate.dtype is dtype
            and w_up.dtype is dtype and w_gate.get_device() == dev and w_up.get_device() == dev
            and x.is_contiguous() and w_gate.is_contiguous() and w_up.is_contiguous()):
        _check_inputs(x, w_gate)  # raises with the reason
        check_like(x, ws, ("w_up", w_up))
    N, K = ws
    if len(xs) == 2:
        return xs[0], K, N, (xs[0], N), _b._dtype_code(x)
    return x.numel() // K if K else 0, K, N, tuple(xs[:-1]) + (N,), _b._dtype_code(x)


def gated_linear_fwd(x, w_gate, w_up, b_gate=None, b_up=None, *, act=ACT_SILU, out=None, pre=None, want_pre=False,
                     workspace=None, stream=None):
    """mamba_gated_linear_fwd on torch tensors: x [..., K], w_gate and w_up
    [N][K], b_gate and b_up [N] float32 or None, out [..., N].  Returns (out,
    pre); pre holds both products, [2, ..., N] float32, which gated_linear_bwd
    takes (None unless want_pre or a buffer for it is given)."""
    import torch
    ts = None if stream is None else _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return gated_linear_fwd(x, w_gate, w_up, b_gate, b_up, act=act, out=out, pre=pre, want_pre=want_pre,
                                    workspace=workspace, stream=ts)
    M, K, N, shape, dt = _check_all(x, w_gate, w_up)
    raw = launch_stream(x, stream)
    if b_gate is not None or b_up is not None:
        check_f32(x, (N,), ("b_gate", b_gate), ("b_up", b_up))
    act = int(act)  # (a tensor would be looked up below by its identity)
    need, _ = _sizes(M, K, N, dt)
    if need == 0 and workspace is None:
        dims = _bare_dims(M, K, N, dt, act)
    else:
        held = make_linear_dims(M, K, N, dt, act=act)
        workspace = use_workspace(held, need, workspace, x)
        dims = ctypes.byref(held)
    if out is None:
        out = x.new_empty(shape)
    else:
        check_like(x, shape, ("out", out))
    if pre is not None:
        check_f32(x, (2,) + shape, ("pre", pre))
    elif want_pre:
        pre = torch.empty((2,) + shape, dtype=torch.float32, device=x.device)
    done(_b.load_library().mamba_gated_linear_fwd(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), ptr(b_gate),
                                                  ptr(b_up), dims, out.data_ptr(), ptr(pre), raw),
         "mamba_gated_linear_fwd")
    return out, pre


def gated_linear_bwd(x, w_gate, w_up, *, dout, pre, act=ACT_SILU, want_dx=True, want_dweight=True, want_dbias=True,
                     workspace=None, stream=None):
    """mamba_gated_linear_bwd on torch tensors, with the pre that
    gated_linear_fwd returned.  Returns a dict with dx, dw_gate, dw_up, db_gate
    and db_up [N] float32 (None unless wanted)."""
    import torch
    ts = None if stream is None else _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return gated_linear_bwd(x, w_gate, w_up, dout=dout, pre=pre, act=act, want_dx=want_dx,
                                    want_dweight=want_dweight, want_dbias=want_dbias, workspace=workspace, stream=ts)
    M, K, N, shape, dt = _check_all(x, w_gate, w_up)
    raw = launch_stream(x, stream)
    check_like(x, shape, ("dout", dout))
    check_f32(x, (2,) + shape, ("pre", pre))
    _, need = _sizes(M, K, N, dt)
    dims = make_linear_dims(M, K, N, dt, act=act)
    workspace = use_workspace(dims, need, workspace, x)
    dx = torch.empty_like(x) if want_dx else None
    dw_gate, dw_up = (torch.empty_like(w_gate), torch.empty_like(w_up)) if want_dweight else (None, None)
    db_gate, db_up = torch.empty((2, N), dtype=torch.float32, device=x.device) if want_dbias else (None, None)
    done(_b.load_library().mamba_gated_linear_bwd(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), ptr(pre),
                                                  dout.data_ptr(), ctypes.byref(dims), ptr(dx), ptr(dw_gate),
                                                  ptr(dw_up), ptr(db_gate), ptr(db_up), raw),
         "mamba_gated_linear_bwd")
    return dict(dx=dx, dw_gate=dw_gate, dw_up=dw_up, db_gate=db_gate, db_up=db_up)

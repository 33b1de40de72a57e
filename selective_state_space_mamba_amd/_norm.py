"""Binding of group normalisation with an activation (mamba_group_norm_*,
include/mamba_scan.h): x [B][L][D] float32 or bfloat16, channels last,
out = act((x - mean)·rstd·weight + bias) over G groups of channels."""
from __future__ import annotations

import ctypes
import functools

from . import _binding as _b
from ._call import check_f32, check_like, done, launch_stream, ptr, query, use_workspace

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3


class NormDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64), ("groups", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("eps", ctypes.c_float),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


def declare(lib):
    vp, dims = ctypes.c_void_p, ctypes.POINTER(NormDims)
    for name in ("fwd_workspace_bytes", "bwd_workspace_bytes"):
        fn = getattr(lib, "mamba_group_norm_" + name)
        fn.restype, fn.argtypes = ctypes.c_size_t, [dims]
    lib.mamba_group_norm_fwd.restype = ctypes.c_int
    lib.mamba_group_norm_fwd.argtypes = [vp] * 3 + [dims] + [vp] * 4
    lib.mamba_group_norm_bwd.restype = ctypes.c_int
    lib.mamba_group_norm_bwd.argtypes = [vp] * 6 + [dims] + [vp] * 4


def make_norm_dims(batch, seqlen, dim, groups, dtype, *, act=ACT_NONE, eps=1e-5, workspace=None,
                   workspace_bytes=0) -> NormDims:
    return NormDims(int(batch), int(seqlen), int(dim), int(groups), int(dtype), int(act), float(eps),
                    _b._ptr(workspace), int(workspace_bytes))


def group_norm_fwd_workspace_bytes(dims: NormDims) -> int:
    return query("mamba_group_norm_fwd_workspace_bytes", dims)


def group_norm_bwd_workspace_bytes(dims: NormDims) -> int:
    return query("mamba_group_norm_bwd_workspace_bytes", dims)


@functools.lru_cache(maxsize=512)
def _sizes(Bsz, L, Dm, groups, dt):
    """(forward, backward) workspace: pure functions of the sizes."""
    d = make_norm_dims(Bsz, L, Dm, groups, dt)
    return group_norm_fwd_workspace_bytes(d), group_norm_bwd_workspace_bytes(d)


def _check_inputs(x, weight, bias):
    if x.dim() != 3:
        raise ValueError("x must be [B][L][D], got %s" % (tuple(x.shape),))
    dt = _b._dtype_code(x)
    shape = x.shape
    check_like(x, shape, ("x", x))
    check_f32(x, shape[2:], ("weight", weight), ("bias", bias))
    return tuple(shape) + (dt,)


def group_norm_fwd(x, groups, weight=None, bias=None, *, eps=1e-5, act=ACT_NONE, out=None, mean=None, rstd=None,
                   workspace=None, stream=None):
    """mamba_group_norm_fwd on torch tensors.  Returns (out [B][L][D], mean
    [B][G], rstd [B][G]); the statistics are what group_norm_bwd takes."""
    import torch
    ts = _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return group_norm_fwd(x, groups, weight, bias, eps=eps, act=act, out=out, mean=mean, rstd=rstd,
                                  workspace=workspace, stream=ts)
    Bsz, L, Dm, dt = _check_inputs(x, weight, bias)
    raw = launch_stream(x, stream)
    groups = int(groups)
    need, _ = _sizes(Bsz, L, Dm, groups, dt)
    dims = make_norm_dims(Bsz, L, Dm, groups, dt, act=act, eps=eps)
    workspace = use_workspace(dims, need, workspace, x)
    if out is None:
        out = torch.empty_like(x)
    else:
        check_like(x, x.shape, ("out", out))
    check_f32(x, (Bsz, groups), ("mean", mean), ("rstd", rstd))
    mean = torch.empty((Bsz, groups), dtype=torch.float32, device=x.device) if mean is None else mean
    rstd = torch.empty_like(mean) if rstd is None else rstd
    done(_b.load_library().mamba_group_norm_fwd(x.data_ptr(), ptr(weight), ptr(bias), ctypes.byref(dims),
                                                out.data_ptr(), mean.data_ptr(), rstd.data_ptr(), raw),
         "mamba_group_norm_fwd")
    return out, mean, rstd


def group_norm_bwd(x, groups, weight=None, bias=None, *, dout, mean, rstd, act=ACT_NONE, workspace=None, stream=None):
    """mamba_group_norm_bwd on torch tensors, with the mean and rstd that
    group_norm_fwd returned for the same arguments.  Returns a dict with dx,
    dweight and dbias (None where the input is None)."""
    import torch
    ts = _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return group_norm_bwd(x, groups, weight, bias, dout=dout, mean=mean, rstd=rstd, act=act,
                                  workspace=workspace, stream=ts)
    Bsz, L, Dm, dt = _check_inputs(x, weight, bias)
    raw = launch_stream(x, stream)
    groups = int(groups)
    _, need = _sizes(Bsz, L, Dm, groups, dt)
    dims = make_norm_dims(Bsz, L, Dm, groups, dt, act=act)
    workspace = use_workspace(dims, need, workspace, x)
    check_like(x, x.shape, ("dout", dout))
    check_f32(x, (Bsz, groups), ("mean", mean), ("rstd", rstd))
    dx = torch.empty_like(x)
    dweight = None if weight is None else torch.empty_like(weight)
    dbias = None if bias is None else torch.empty_like(bias)
    done(_b.load_library().mamba_group_norm_bwd(x.data_ptr(), ptr(weight), ptr(bias), dout.data_ptr(),
                                                mean.data_ptr(), rstd.data_ptr(), ctypes.byref(dims), dx.data_ptr(),
                                                ptr(dweight), ptr(dbias), raw), "mamba_group_norm_bwd")
    return dict(dx=dx, dweight=dweight, dbias=dbias)

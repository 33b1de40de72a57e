"""Binding of group normalisation with an activation (mamba_group_norm_*,
include/mamba_scan.h): x [B][L][D] float32 or bfloat16, channels last,
out = act((x - mean)·rstd·weight + bias) over G groups of channels."""
from __future__ import annotations

import ctypes

from . import _binding as _b
from ._glr import _query, _workspace

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
    return _query("mamba_group_norm_fwd_workspace_bytes", dims)


def group_norm_bwd_workspace_bytes(dims: NormDims) -> int:
    return _query("mamba_group_norm_bwd_workspace_bytes", dims)


def _check_inputs(x, weight, bias):
    import torch
    if x.dim() != 3:
        raise ValueError("x must be [B][L][D], got %s" % (tuple(x.shape),))
    _b._check(x, "x", tuple(x.shape), x.dtype, x.device)
    _b._check(weight, "weight", (x.shape[2],), torch.float32, x.device)
    _b._check(bias, "bias", (x.shape[2],), torch.float32, x.device)
    return tuple(x.shape) + (_b._dtype_code(x), x.device)


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
    lib = _b.load_library()
    Bsz, L, Dm, dt, dev = _check_inputs(x, weight, bias)
    dims = make_norm_dims(Bsz, L, Dm, groups, dt, act=act, eps=eps)
    workspace = _workspace(dims, group_norm_fwd_workspace_bytes(dims), workspace, dev)
    out = torch.empty_like(x) if out is None else out
    _b._check(out, "out", (Bsz, L, Dm), x.dtype, dev)
    mean = torch.empty((Bsz, groups), dtype=torch.float32, device=dev) if mean is None else mean
    rstd = torch.empty((Bsz, groups), dtype=torch.float32, device=dev) if rstd is None else rstd
    _b._check(mean, "mean", (Bsz, groups), torch.float32, dev)
    _b._check(rstd, "rstd", (Bsz, groups), torch.float32, dev)
    rc = lib.mamba_group_norm_fwd(_b._ptr(x), _b._ptr(weight), _b._ptr(bias), ctypes.byref(dims), _b._ptr(out),
                                  _b._ptr(mean), _b._ptr(rstd), _b._stream(stream))
    if rc != _b.MAMBA_OK:
        raise _b.MambaError(rc, "mamba_group_norm_fwd")
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
    lib = _b.load_library()
    Bsz, L, Dm, dt, dev = _check_inputs(x, weight, bias)
    dims = make_norm_dims(Bsz, L, Dm, groups, dt, act=act)
    workspace = _workspace(dims, group_norm_bwd_workspace_bytes(dims), workspace, dev)
    _b._check(dout, "dout", (Bsz, L, Dm), x.dtype, dev)
    _b._check(mean, "mean", (Bsz, groups), torch.float32, dev)
    _b._check(rstd, "rstd", (Bsz, groups), torch.float32, dev)
    g = dict(dx=torch.empty_like(x), dweight=None if weight is None else torch.empty_like(weight),
             dbias=None if bias is None else torch.empty_like(bias))
    rc = lib.mamba_group_norm_bwd(_b._ptr(x), _b._ptr(weight), _b._ptr(bias), _b._ptr(dout), _b._ptr(mean),
                                  _b._ptr(rstd), ctypes.byref(dims), _b._ptr(g["dx"]), _b._ptr(g["dweight"]),
                                  _b._ptr(g["dbias"]), _b._stream(stream))
    if rc != _b.MAMBA_OK:
        raise _b.MambaError(rc, "mamba_group_norm_bwd")
    return g

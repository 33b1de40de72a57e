"""Binding of the gated linear recurrence (mamba_glr_*, include/mamba_scan.h).

    a = exp(-scale·softplus(lam)·sigmoid(r))          (lam None: a = sigmoid(r))
    h = a·h + beta·sigmoid(i)·x,  beta = sqrt(1 - a²) | 1 - a | 1
    out = h·silu(z)

x, r, i, z [B][L][D] float32 or bfloat16 (i and z may be None), lam [D] float32
or None, the state [B][D] float32.
"""
from __future__ import annotations

import ctypes

from . import _binding as _b

GLR_SQRT, GLR_LERP, GLR_UNIT = 0, 1, 2


class GlrDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("dim", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("input_rule", ctypes.c_int32), ("reverse", ctypes.c_int32),
        ("scale", ctypes.c_float), ("initial_state", ctypes.c_void_p), ("reset", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


def declare(lib):
    vp, i32, sz, dims = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(GlrDims)
    for name in ("fwd_workspace_bytes", "bwd_workspace_bytes", "saved_bytes"):
        fn = getattr(lib, "mamba_glr_" + name)
        fn.restype, fn.argtypes = sz, [dims]
    lib.mamba_glr_fwd.restype = i32
    lib.mamba_glr_fwd.argtypes = [vp] * 5 + [dims] + [vp] * 3 + [sz, vp]
    lib.mamba_glr_bwd.restype = i32
    lib.mamba_glr_bwd.argtypes = [vp] * 7 + [dims] + [vp] * 7 + [sz, vp]
    lib.mamba_glr_step.restype = i32
    lib.mamba_glr_step.argtypes = [vp] * 6 + [dims, vp, vp]


def make_glr_dims(batch, seqlen, dim, dtype, *, input_rule=GLR_SQRT, reverse=False, scale=8.0, initial_state=None,
                  reset=None, workspace=None, workspace_bytes=0) -> GlrDims:
    return GlrDims(int(batch), int(seqlen), int(dim), int(dtype), int(input_rule), 1 if reverse else 0, float(scale),
                   _b._ptr(initial_state), _b._ptr(reset), _b._ptr(workspace), int(workspace_bytes))


def _query(name, dims) -> int:
    n = getattr(_b.load_library(), name)(ctypes.byref(dims))
    if n == ctypes.c_size_t(-1).value:
        raise _b.MambaError(_b.MAMBA_ERR_UNSUPPORTED, name)
    return n


def glr_fwd_workspace_bytes(dims: GlrDims) -> int:
    return _query("mamba_glr_fwd_workspace_bytes", dims)


def glr_bwd_workspace_bytes(dims: GlrDims) -> int:
    return _query("mamba_glr_bwd_workspace_bytes", dims)


def glr_saved_bytes(dims: GlrDims) -> int:
    return _query("mamba_glr_saved_bytes", dims)


def _bytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _workspace(dims, need, workspace, dev):
    """Puts a workspace of need bytes (the caller's, if it is large enough) into dims and returns it, to be kept
    until the launch."""
    import torch
    _b._check_buffer(workspace, "workspace", dev)
    if need > 0 and _bytes(workspace) < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if need > 0:
        dims.workspace, dims.workspace_bytes = workspace.data_ptr(), _bytes(workspace)
    return workspace


def _check_inputs(x, r, i, z, lam, initial_state, reset):
    import torch
    if x.dim() != 3:
        raise ValueError("x must be [B][L][D], got %s" % (tuple(x.shape),))
    Bsz, L, Dm = x.shape
    dev, tdt = x.device, x.dtype
    for name, t in (("x", x), ("r", r), ("i", i), ("z", z)):
        _b._check(t, name, (Bsz, L, Dm), tdt, dev)
    _b._check(lam, "lam", (Dm,), torch.float32, dev)
    _b._check(initial_state, "initial_state", (Bsz, Dm), torch.float32, dev)
    if reset is not None:
        _b._check(reset, "reset", (Bsz, L), torch.bool if reset.dtype == torch.bool else torch.uint8, dev)
    return Bsz, L, Dm, _b._dtype_code(x), dev


def glr_fwd(x, r, i=None, z=None, lam=None, *, scale=8.0, input_rule=GLR_SQRT, reverse=False, initial_state=None,
            reset=None, out=None, last_state=None, want_last_state=True, workspace=None, stream=None):
    """mamba_glr_fwd on torch tensors.  reset: [B][L] uint8 or bool, nonzero
    where a token starts a new sequence.  Returns (out [B][L][D], last_state
    [B][D] or None)."""
    out, last_state, _ = _fwd(x, r, i, z, lam, scale, input_rule, reverse, initial_state, reset, out, last_state,
                              want_last_state, workspace, stream, False, None)
    return out, last_state


def glr_fwd_save(x, r, i=None, z=None, lam=None, *, scale=8.0, input_rule=GLR_SQRT, reverse=False,
                 initial_state=None, reset=None, out=None, last_state=None, want_last_state=True, workspace=None,
                 saved=None, stream=None):
    """glr_fwd that also returns the states glr_bwd(..., saved=...) reads in
    place of recomputing them: (out, last_state, saved)."""
    return _fwd(x, r, i, z, lam, scale, input_rule, reverse, initial_state, reset, out, last_state, want_last_state,
                workspace, stream, True, saved)


def _fwd(x, r, i, z, lam, scale, input_rule, reverse, initial_state, reset, out, last_state, want_last_state,
         workspace, stream, save, saved):
    import torch
    ts = _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return _fwd(x, r, i, z, lam, scale, input_rule, reverse, initial_state, reset, out, last_state,
                        want_last_state, workspace, ts, save, saved)
    lib = _b.load_library()
    Bsz, L, Dm, dt, dev = _check_inputs(x, r, i, z, lam, initial_state, reset)
    if out is None:
        out = torch.empty_like(x)
    _b._check(out, "out", (Bsz, L, Dm), x.dtype, dev)
    if last_state is None and want_last_state:
        last_state = torch.empty((Bsz, Dm), dtype=torch.float32, device=dev)
    _b._check(last_state, "last_state", (Bsz, Dm), torch.float32, dev)
    dims = make_glr_dims(Bsz, L, Dm, dt, input_rule=input_rule, reverse=reverse, scale=scale,
                         initial_state=initial_state, reset=reset)
    workspace = _workspace(dims, glr_fwd_workspace_bytes(dims), workspace, dev)
    _b._check_buffer(saved, "saved", dev)
    if save and saved is None:
        saved = torch.empty(glr_saved_bytes(dims), dtype=torch.uint8, device=dev)
    rc = lib.mamba_glr_fwd(_b._ptr(x), _b._ptr(r), _b._ptr(i), _b._ptr(z), _b._ptr(lam), ctypes.byref(dims),
                           _b._ptr(out), _b._ptr(last_state), _b._ptr(saved), _bytes(saved), _b._stream(stream))
    if rc != _b.MAMBA_OK:
        raise _b.MambaError(rc, "mamba_glr_fwd")
    return out, last_state, saved


def glr_bwd(x, r, i=None, z=None, lam=None, *, dout, dlast=None, scale=8.0, input_rule=GLR_SQRT, reverse=False,
            initial_state=None, reset=None, workspace=None, saved=None, stream=None):
    """mamba_glr_bwd on torch tensors: gradients of sum(dout·out) +
    sum(dlast·last_state) for the glr_fwd call with the same arguments.  Returns
    a dict with dx, dr, di, dz, dlam (None where the input is None) and dinit
    [B][D].  saved: what glr_fwd_save returned, or None to recompute the states."""
    import torch
    ts = _b._foreign_stream(stream)
    if ts is not None:
        with torch.cuda.stream(ts):
            return glr_bwd(x, r, i, z, lam, dout=dout, dlast=dlast, scale=scale, input_rule=input_rule,
                           reverse=reverse, initial_state=initial_state, reset=reset, workspace=workspace,
                           saved=saved, stream=ts)
    lib = _b.load_library()
    Bsz, L, Dm, dt, dev = _check_inputs(x, r, i, z, lam, initial_state, reset)
    _b._check(dout, "dout", (Bsz, L, Dm), x.dtype, dev)
    _b._check(dlast, "dlast", (Bsz, Dm), torch.float32, dev)
    g = dict(dx=torch.empty_like(x), dr=torch.empty_like(x), di=None if i is None else torch.empty_like(x),
             dz=None if z is None else torch.empty_like(x), dlam=None if lam is None else torch.empty_like(lam),
             dinit=torch.empty((Bsz, Dm), dtype=torch.float32, device=dev))
    dims = make_glr_dims(Bsz, L, Dm, dt, input_rule=input_rule, reverse=reverse, scale=scale,
                         initial_state=initial_state, reset=reset)
    workspace = _workspace(dims, glr_bwd_workspace_bytes(dims), workspace, dev)
    _b._check_buffer(saved, "saved", dev)
    rc = lib.mamba_glr_bwd(_b._ptr(x), _b._ptr(r), _b._ptr(i), _b._ptr(z), _b._ptr(lam), _b._ptr(dout),
                           _b._ptr(dlast), ctypes.byref(dims), _b._ptr(g["dx"]), _b._ptr(g["dr"]), _b._ptr(g["di"]),
                           _b._ptr(g["dz"]), _b._ptr(g["dlam"]), _b._ptr(g["dinit"]), _b._ptr(saved), _bytes(saved),
                           _b._stream(stream))
    if rc != _b.MAMBA_OK:
        raise _b.MambaError(rc, "mamba_glr_bwd")
    return g


def glr_step(state, x_t, r_t, i_t=None, z_t=None, lam=None, *, scale=8.0, input_rule=GLR_SQRT, out=None, stream=None):
    """mamba_glr_step on torch tensors: state [B][D] float32 (updated in
    place), x_t/r_t/i_t/z_t [B][D].  Returns out [B][D]."""
    import torch
    ts = _b._foreign_stream(stream) if out is None else None
    if ts is not None:
        with torch.cuda.stream(ts):
            return glr_step(state, x_t, r_t, i_t, z_t, lam, scale=scale, input_rule=input_rule, out=out, stream=ts)
    lib = _b.load_library()
    if x_t.dim() != 2:
        raise ValueError("x_t must be [B][D], got %s" % (tuple(x_t.shape),))
    Bsz, Dm = shape = x_t.shape
    dev, tdt = x_t.device, x_t.dtype
    _b._check(state, "state", shape, torch.float32, dev)
    for name, t in (("x_t", x_t), ("r_t", r_t), ("i_t", i_t), ("z_t", z_t)):
        _b._check(t, name, shape, tdt, dev)
    _b._check(lam, "lam", (Dm,), torch.float32, dev)
    if out is None:
        out = torch.empty_like(x_t)
    _b._check(out, "out", shape, tdt, dev)
    dims = make_glr_dims(Bsz, 1, Dm, _b._dtype_code(x_t), input_rule=input_rule, scale=scale)
    rc = lib.mamba_glr_step(_b._ptr(state), _b._ptr(x_t), _b._ptr(r_t), _b._ptr(i_t), _b._ptr(z_t), _b._ptr(lam),
                            ctypes.byref(dims), _b._ptr(out), _b._stream(stream))
    if rc != _b.MAMBA_OK:
        raise _b.MambaError(rc, "mamba_glr_step")
    return out

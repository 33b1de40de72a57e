"""Binding of the gated linear recurrence (mamba_glr_*, include/mamba_scan.h).

    a = exp(-scale·softplus(lam)·sigmoid(r))          (lam None: a = sigmoid(r))
    h = a·h + beta·sigmoid(i)·x,  beta = sqrt(1 - a²) | 1 - a | 1
    out = h·silu(z)

x, r, i, z [B][L][D] float32 or bfloat16 (i and z may be None), lam [D] float32
or None, the state [B][D] float32.
"""
from __future__ import annotations

import ctypes
import functools

from . import _binding as _b
from ._call import check_f32, check_like, done, launch_stream, nbytes, ptr, query, use_workspace

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


def glr_fwd_workspace_bytes(dims: GlrDims) -> int:
    return query("mamba_glr_fwd_workspace_bytes", dims)


def glr_bwd_workspace_bytes(dims: GlrDims) -> int:
    return query("mamba_glr_bwd_workspace_bytes", dims)


def glr_saved_bytes(dims: GlrDims) -> int:
    return query("mamba_glr_saved_bytes", dims)


@functools.lru_cache(maxsize=512)
def _sizes(Bsz, L, Dm, dt):
    """(forward workspace, backward workspace, saved states): pure functions of the sizes."""
    d = make_glr_dims(Bsz, L, Dm, dt)
    return glr_fwd_workspace_bytes(d), glr_bwd_workspace_bytes(d), glr_saved_bytes(d)


def _check_inputs(x, r, i, z, lam, initial_state, reset):
    import torch
    if x.dim() != 3:
        raise ValueError("x must be [B][L][D], got %s" % (tuple(x.shape),))
    dt = _b._dtype_code(x)
    shape = x.shape
    Bsz, L, Dm = shape
    check_like(x, shape, ("x", x), ("r", r), ("i", i), ("z", z))
    if lam is not None:
        check_f32(x, (Dm,), ("lam", lam))
    if initial_state is not None:
        check_f32(x, (Bsz, Dm), ("initial_state", initial_state))
    if reset is not None:
        _b._check(reset, "reset", (Bsz, L), torch.bool if reset.dtype == torch.bool else torch.uint8, x.device)
    return Bsz, L, Dm, dt


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
    Bsz, L, Dm, dt = _check_inputs(x, r, i, z, lam, initial_state, reset)
    raw = launch_stream(x, stream)
    need, _, need_saved = _sizes(Bsz, L, Dm, dt)
    if out is None:
        out = torch.empty_like(x)
    else:
        check_like(x, x.shape, ("out", out))
    if last_state is not None:
        check_f32(x, (Bsz, Dm), ("last_state", last_state))
    elif want_last_state:
        last_state = torch.empty((Bsz, Dm), dtype=torch.float32, device=x.device)
    dims = make_glr_dims(Bsz, L, Dm, dt, input_rule=input_rule, reverse=reverse, scale=scale,
                         initial_state=initial_state, reset=reset)
    workspace = use_workspace(dims, need, workspace, x)
    if saved is not None:
        _b._check_buffer(saved, "saved", x.device)
    elif save:
        saved = torch.empty(need_saved, dtype=torch.uint8, device=x.device)
    done(_b.load_library().mamba_glr_fwd(x.data_ptr(), r.data_ptr(), ptr(i), ptr(z), ptr(lam), ctypes.byref(dims),
                                         out.data_ptr(), ptr(last_state), ptr(saved), nbytes(saved), raw),
         "mamba_glr_fwd")
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
    Bsz, L, Dm, dt = _check_inputs(x, r, i, z, lam, initial_state, reset)
    raw = launch_stream(x, stream)
    check_like(x, x.shape, ("dout", dout))
    if dlast is not None:
        check_f32(x, (Bsz, Dm), ("dlast", dlast))
    _, need, _ = _sizes(Bsz, L, Dm, dt)
    dx, dr = torch.empty_like(x), torch.empty_like(x)
    di = None if i is None else torch.empty_like(x)
    dz = None if z is None else torch.empty_like(x)
    dlam = None if lam is None else torch.empty_like(lam)
    dinit = torch.empty((Bsz, Dm), dtype=torch.float32, device=x.device)
    dims = make_glr_dims(Bsz, L, Dm, dt, input_rule=input_rule, reverse=reverse, scale=scale,
                         initial_state=initial_state, reset=reset)
    workspace = use_workspace(dims, need, workspace, x)
    _b._check_buffer(saved, "saved", x.device)
    done(_b.load_library().mamba_glr_bwd(x.data_ptr(), r.data_ptr(), ptr(i), ptr(z), ptr(lam), dout.data_ptr(),
                                         ptr(dlast), ctypes.byref(dims), dx.data_ptr(), dr.data_ptr(), ptr(di),
                                         ptr(dz), ptr(dlam), dinit.data_ptr(), ptr(saved), nbytes(saved), raw),
         "mamba_glr_bwd")
    return dict(dx=dx, dr=dr, di=di, dz=dz, dlam=dlam, dinit=dinit)


@functools.lru_cache(maxsize=512)
def _step_dims(Bsz, Dm, dt, input_rule, scale):
    """The dims of a step hold no pointers and are only read: one for all calls of these sizes.  (Plain numbers as
    arguments: a tensor would be looked up by its identity, whatever it holds by then.)"""
    d = make_glr_dims(Bsz, 1, Dm, dt, input_rule=input_rule, scale=scale)
    return d, ctypes.byref(d)


def glr_step(state, x_t, r_t, i_t=None, z_t=None, lam=None, *, scale=8.0, input_rule=GLR_SQRT, out=None, stream=None):
    """mamba_glr_step on torch tensors: state [B][D] float32 (updated in
    place), x_t/r_t/i_t/z_t [B][D].  Returns out [B][D]."""
    import torch
    ts = _b._foreign_stream(stream) if out is None else None
    if ts is not None:
        with torch.cuda.stream(ts):
            return glr_step(state, x_t, r_t, i_t, z_t, lam, scale=scale, input_rule=input_rule, out=out, stream=ts)
    if x_t.dim() != 2:
        raise ValueError("x_t must be [B][D], got %s" % (tuple(x_t.shape),))
    dt = _b._dtype_code(x_t)
    shape = x_t.shape
    check_like(x_t, shape, ("x_t", x_t), ("r_t", r_t), ("i_t", i_t), ("z_t", z_t), ("out", out))
    check_f32(x_t, shape, ("state", state))
    check_f32(x_t, shape[1:], ("lam", lam))
    raw = launch_stream(x_t, stream)
    if out is None:
        out = torch.empty_like(x_t)
    done(_b.load_library().mamba_glr_step(state.data_ptr(), x_t.data_ptr(), r_t.data_ptr(), ptr(i_t), ptr(z_t),
                                          ptr(lam), _step_dims(shape[0], shape[1], dt, int(input_rule), float(scale))[1],
                                          out.data_ptr(), raw), "mamba_glr_step")
    return out

"""What the bindings of the operators around the scan share: argument checks
that cost little where they pass (a decode step is a few microseconds of GPU
time), the launch stream, workspaces and size queries."""
from __future__ import annotations

import ctypes

from . import _binding as _b


def _raw_current():
    """device -> torch's current stream there as a raw handle.  torch.cuda's own
    way makes a Stream object (1.1 us of a 10 us call); torch._C has the handle alone."""
    import torch
    return getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _device():
    """-> the current device's index.  torch.cuda's own way asks first whether
    there is a GPU in use (0.2 us more); a tensor on one says so."""
    import torch
    return getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


# (both of the above): one name, so that a thread sees both or neither while another makes them
_torch_calls = None


def launch_stream(x, stream) -> int:
    """The raw stream to launch on (torch's current one where stream is None).
    x has to be on the current GPU: that is the device the library launches on."""
    global _torch_calls
    dev = x.get_device()
    if dev < 0 or not x.is_cuda:
        raise ValueError("x is on %s, a GPU is needed" % x.device)
    if _torch_calls is None:
        _torch_calls = _raw_current(), _device()
    current, current_device = _torch_calls
    if dev != current_device():
        raise ValueError("x is on cuda:%d, the current device is cuda:%d" % (dev, current_device()))
    if stream is None:
        return current(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def check_like(x, shape, *named):
    """Each (name, tensor or None) has this shape, and x's type and device, and is contiguous."""
    dtype, dev = x.dtype, x.get_device()
    for name, t in named:
        if t is not None and not (t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev):
            _b._check(t, name, shape, dtype, x.device)  # raises with the reason


def check_f32(x, shape, *named):
    """The same for float32 tensors beside x."""
    import torch
    f32, dev = torch.float32, x.get_device()
    for name, t in named:
        if t is not None and not (t.shape == shape and t.dtype is f32 and t.is_contiguous() and t.get_device() == dev):
            _b._check(t, name, shape, f32, x.device)


def ptr(t):
    return None if t is None else t.data_ptr()


def nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def query(name, dims) -> int:
    n = getattr(_b.load_library(), name)(ctypes.byref(dims))
    if n == ctypes.c_size_t(-1).value:
        raise _b.MambaError(_b.MAMBA_ERR_UNSUPPORTED, name)
    return n


def use_workspace(dims, need, workspace, x):
    """Puts a workspace of need bytes (the caller's, if it is large enough) into
    dims and returns it, to be kept until the launch."""
    import torch
    _b._check_buffer(workspace, "workspace", x.device)
    if need > 0:
        if nbytes(workspace) < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        dims.workspace, dims.workspace_bytes = workspace.data_ptr(), nbytes(workspace)
    return workspace


def done(rc, name):
    if rc != _b.MAMBA_OK:
        raise _b.MambaError(rc, name)

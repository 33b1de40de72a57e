"""MI355X-native (gfx950) selective-scan library.

The compute path is libmamba_scan.so: hand-written HIP kernels behind the C
ABI declared in include/mamba_scan.h.  This package holds its sources
(csrc/), the in-tree build step (build.py), a ctypes binding that only
marshals arguments (_binding.py for the scan, _glr.py for the gated recurrence,
_norm.py for the group normalisation, _linear.py for the matrix product, _rms.py for
the root-mean-square norm, _gated.py for the gated pair of products, _quant.py for
the products with quantised weights, _call.py for what those share), and the seeded input generator used by the tests and
the benchmark (inputs.py).
"""
from ._binding import (DIR_BIDIR, DIR_BWD, DIR_CROSS2D, DIR_FWD, DTYPE_BF16, DTYPE_F32, EXPORTED, LIB_PATH,
                       MambaDims, MambaError, ScanStepper, bwd_workspace_bytes, conv1d_silu, load_library, make_dims, num_dirs,
                       saved_bytes, scan_bwd, scan_fwd, scan_fwd_noalloc, scan_fwd_save, scan_step, status_string, workspace_bytes)
from ._glr import (GLR_LERP, GLR_SQRT, GLR_UNIT, GlrDims, glr_bwd, glr_bwd_workspace_bytes, glr_fwd, glr_fwd_save,
                   glr_fwd_workspace_bytes, glr_saved_bytes, glr_step, make_glr_dims)
from ._linear import (LinearDims, linear_bwd, linear_bwd_workspace_bytes, linear_fwd, linear_fwd_workspace_bytes,
                      linear_plan, make_linear_dims)
from ._norm import (ACT_GELU, ACT_NONE, ACT_RELU, ACT_SILU, NormDims, group_norm_bwd, group_norm_bwd_workspace_bytes,
                    group_norm_fwd, group_norm_fwd_workspace_bytes, make_norm_dims)
from ._gated import gated_linear_bwd, gated_linear_bwd_workspace_bytes, gated_linear_fwd, gated_linear_fwd_workspace_bytes
from ._quant import Q4Dims, linear_q4, linear_q8, linear_q8_workspace_bytes, make_q4_dims
from ._rms import RmsDims, make_rms_dims, rms_norm_bwd, rms_norm_bwd_workspace_bytes, rms_norm_fwd, rms_norm_q8

__all__ = ["DIR_BIDIR", "DIR_BWD", "DIR_CROSS2D", "DIR_FWD", "DTYPE_BF16", "DTYPE_F32", "EXPORTED", "LIB_PATH",
           "MambaDims", "MambaError", "ScanStepper", "bwd_workspace_bytes", "conv1d_silu", "load_library", "make_dims", "num_dirs",
           "saved_bytes", "scan_bwd", "scan_fwd", "scan_fwd_noalloc", "scan_fwd_save", "scan_step", "status_string", "workspace_bytes",
           "GLR_LERP", "GLR_SQRT", "GLR_UNIT", "GlrDims", "glr_bwd", "glr_bwd_workspace_bytes", "glr_fwd", "glr_fwd_save",
           "glr_fwd_workspace_bytes", "glr_saved_bytes", "glr_step", "make_glr_dims",
           "ACT_GELU", "ACT_NONE", "ACT_RELU", "ACT_SILU", "NormDims", "group_norm_bwd", "group_norm_bwd_workspace_bytes",
           "group_norm_fwd", "group_norm_fwd_workspace_bytes", "make_norm_dims",
           "LinearDims", "linear_bwd", "linear_bwd_workspace_bytes", "linear_fwd", "linear_fwd_workspace_bytes", "linear_plan", "make_linear_dims",
           "RmsDims", "make_rms_dims", "rms_norm_bwd", "rms_norm_bwd_workspace_bytes", "rms_norm_fwd", "rms_norm_q8",
           "gated_linear_bwd", "gated_linear_bwd_workspace_bytes", "gated_linear_fwd", "gated_linear_fwd_workspace_bytes",
           "Q4Dims", "linear_q4", "linear_q8", "linear_q8_workspace_bytes", "make_q4_dims"]

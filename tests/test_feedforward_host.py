"""Host-side checks of the feed-forward layer's operators (no GPU work): sizes,
refusals before any launch, and the float64 references' gradients against
differences."""
import ctypes
import os

import pytest

import selective_state_space_mamba_amd as ms
from selective_state_space_mamba_amd import _binding as E

from ffutil import maker, rms_grads, rms_ref

FAKE = 0x100000  # 16-byte aligned stand-in pointer: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ms.LIB_PATH):
        from selective_state_space_mamba_amd import build
        build.build(force=False)
    return ms.load_library()


def rms_dims(**kw):
    base = dict(rows=100, dim=64, dtype=ms.DTYPE_BF16)
    base.update(kw)
    return ms.make_rms_dims(base.pop("rows"), base.pop("dim"), base.pop("dtype"), **base)


RMS_BAD = [(dict(rows=0), E.MAMBA_ERR_INVALID), (dict(dim=0), E.MAMBA_ERR_INVALID), (dict(dim=-8), E.MAMBA_ERR_INVALID),
           (dict(dtype=2), E.MAMBA_ERR_INVALID), (dict(residual_dtype=5), E.MAMBA_ERR_INVALID),
           (dict(eps=-1.0), E.MAMBA_ERR_INVALID), (dict(eps=float("nan")), E.MAMBA_ERR_INVALID),
           (dict(eps=float("inf")), E.MAMBA_ERR_INVALID), (dict(dim=16385), E.MAMBA_ERR_UNSUPPORTED),
           (dict(rows=(1 << 36) + 1), E.MAMBA_ERR_UNSUPPORTED),
           (dict(dtype=ms.DTYPE_F32, residual_dtype=ms.DTYPE_BF16), E.MAMBA_ERR_UNSUPPORTED)]


def test_rms_sizes(lib):
    assert ms.rms_norm_bwd_workspace_bytes(rms_dims()) == 25 * 64 * 4
    assert ms.rms_norm_bwd_workspace_bytes(rms_dims(rows=1 << 30)) == 1024 * 64 * 4
    for bad, _ in RMS_BAD:
        with pytest.raises(ms.MambaError):
            ms.rms_norm_bwd_workspace_bytes(rms_dims(**bad))


def test_rms_refusals(lib):
    def fwd(d, x=FAKE, res=None, w=None, out=FAKE, added=None, rstd=None):
        return lib.mamba_rms_norm_fwd(x, res, w, d and ctypes.byref(d), out, added, rstd, None)

    def q8(d, x=FAKE, res=None, w=None, out=FAKE, scale=FAKE, added=None):
        return lib.mamba_rms_norm_q8(x, res, w, d and ctypes.byref(d), out, scale, added, None)

    def bwd(d, s=FAKE, w=FAKE, rstd=FAKE, dout=FAKE, dadded=None, dx=FAKE, dres=None, dw=None):
        return lib.mamba_rms_norm_bwd(s, w, rstd, dout, dadded, d and ctypes.byref(d), dx, dres, dw, None)

    for call, needed in ((fwd, ("x", "out")), (q8, ("x", "out", "scale")), (bwd, ("s", "rstd", "dout", "dx"))):
        assert call(None) == E.MAMBA_ERR_INVALID
        for miss in needed:
            assert call(rms_dims(), **{miss: None}) == E.MAMBA_ERR_INVALID
        for bad, code in RMS_BAD:
            assert call(rms_dims(**bad)) == code, bad
    for call, odd in ((fwd, ("x", "res", "out", "added")), (q8, ("x", "res", "added")), (bwd, ("s", "dout", "dadded", "dx", "dres"))):
        for k in odd:
            assert call(rms_dims(), **{k: FAKE + 1}) == E.MAMBA_ERR_UNSUPPORTED, (call, k)
    for call, odd in ((fwd, ("w", "rstd")), (q8, ("w", "scale")), (bwd, ("w", "rstd", "dw"))):
        for k in odd:
            assert call(rms_dims(), **{k: FAKE + 2}) == E.MAMBA_ERR_UNSUPPORTED, (call, k)
    assert fwd(rms_dims(residual_dtype=ms.DTYPE_F32), res=FAKE + 2) == E.MAMBA_ERR_UNSUPPORTED
    assert bwd(rms_dims(), dw=FAKE) == E.MAMBA_ERR_WORKSPACE
    need = ms.rms_norm_bwd_workspace_bytes(rms_dims())
    assert bwd(rms_dims(workspace=FAKE, workspace_bytes=need - 1), dw=FAKE) == E.MAMBA_ERR_WORKSPACE
    assert bwd(rms_dims(workspace=FAKE + 8, workspace_bytes=need), dw=FAKE) == E.MAMBA_ERR_UNSUPPORTED


def test_rms_reference_gradients_against_differences():
    """Central differences in float64: 1e-7 is asked, of 1e-10 + 1e-16/eps."""
    n = maker(3, "cpu")
    x, w, dout, dadded = (n(s).double() for s in ((4, 13), (13,), (4, 13), (4, 13)))

    def loss(x, w):
        _, _, y = rms_ref(x, w, None, 1e-5)
        return float((y * dout).sum() + (x * dadded).sum())

    _, rstd, _ = rms_ref(x, w, None, 1e-5)
    ds, _, dw, _ = rms_grads(x, w, rstd, dout, dadded)
    eps = 1e-5
    for k, g in (("x", ds), ("w", dw)):
        v = dict(x=x, w=w)
        d = n(tuple(g.shape)).double()
        num = (loss(**dict(v, **{k: v[k] + eps * d})) - loss(**dict(v, **{k: v[k] - eps * d}))) / (2 * eps)
        want = float((g * d).sum())
        assert abs(num - want) <= 1e-7 * max(1.0, abs(want)), (k, num, want)

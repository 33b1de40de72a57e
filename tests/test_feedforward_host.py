"""Host-side checks of the feed-forward layer's operators (no GPU work): sizes,
refusals before any launch, and the float64 references' gradients against
differences."""
import ctypes
import os
import random

import pytest

import selective_state_space_mamba_amd as ms
from selective_state_space_mamba_amd import _binding as E

from ffutil import gated_ref, maker, planned, planned_kind, rms_grads, rms_ref

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
    assert ms.rms_norm_bwd_workspace_bytes(rms_dims()) == 0  # few rows: no scratch
    assert ms.rms_norm_bwd_workspace_bytes(rms_dims(rows=1024)) == 0
    assert ms.rms_norm_bwd_workspace_bytes(rms_dims(rows=1025)) == 33 * 64 * 4
    assert ms.rms_norm_bwd_workspace_bytes(rms_dims(rows=1 << 30)) == 1024 * 64 * 4
    assert ms.rms_norm_bwd_workspace_bytes(rms_dims(rows=1 << 30, dim=512)) == 512 * 512 * 4
    for bad, _ in RMS_BAD:
        with pytest.raises(ms.MambaError):
            ms.rms_norm_bwd_workspace_bytes(rms_dims(**bad))


def test_planned_tiles(lib):
    """The tests' rule for tiles and shares is the library's: the plain product's own report, the others' workspaces."""
    rng = random.Random(6)
    seen = set()
    for _ in range(1500):
        M, N, K = (int(2 ** rng.uniform(a, b)) for a, b in ((6.1, 16), (0, 11), (1, 11)))
        N, K = 8 * N, 8 * K
        d = ms.make_linear_dims(M, K, N, ms.DTYPE_BF16)
        assert planned(M, N, K)[:3] == tuple(ms.linear_plan(d, 0)), (M, N, K)
        for op, query, cols, k in (("gated", ms.gated_linear_fwd_workspace_bytes, 2 * N, K),
                                   ("q8", ms.linear_q8_workspace_bytes, N, 2 * K)):
            kind = planned_kind(op, M, k, N)
            shares = kind[3] if kind[0] == "tile" else 1
            need = -(-shares * M * cols * 4 // 256) * 256 if shares > 1 else 0
            assert query(ms.make_linear_dims(M, k, N, ms.DTYPE_BF16)) == need, (op, M, N, k)
            seen.add((op, kind[0], shares > 1))
    assert len(seen) == 8, seen


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
    assert bwd(rms_dims(rows=1100), dw=FAKE) == E.MAMBA_ERR_WORKSPACE
    need = ms.rms_norm_bwd_workspace_bytes(rms_dims(rows=1100))
    assert bwd(rms_dims(rows=1100, workspace=FAKE, workspace_bytes=need - 1), dw=FAKE) == E.MAMBA_ERR_WORKSPACE
    assert bwd(rms_dims(rows=1100, workspace=FAKE + 8, workspace_bytes=need), dw=FAKE) == E.MAMBA_ERR_UNSUPPORTED


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


def linear_dims(**kw):
    base = dict(rows=100, in_dim=64, out_dim=32, dtype=ms.DTYPE_BF16)
    base.update(kw)
    return ms.make_linear_dims(base.pop("rows"), base.pop("in_dim"), base.pop("out_dim"), base.pop("dtype"), **base)


LINEAR_BAD = [(dict(rows=0), E.MAMBA_ERR_INVALID), (dict(in_dim=0), E.MAMBA_ERR_INVALID), (dict(out_dim=-8), E.MAMBA_ERR_INVALID),
              (dict(dtype=2), E.MAMBA_ERR_INVALID), (dict(act=4), E.MAMBA_ERR_INVALID), (dict(in_dim=12), E.MAMBA_ERR_UNSUPPORTED),
              (dict(out_dim=20), E.MAMBA_ERR_UNSUPPORTED), (dict(in_dim=(1 << 20) + 16), E.MAMBA_ERR_UNSUPPORTED),
              (dict(rows=(1 << 29) + 1), E.MAMBA_ERR_UNSUPPORTED)]


def test_gated_sizes(lib):
    assert ms.gated_linear_fwd_workspace_bytes(linear_dims()) == 0
    assert ms.gated_linear_fwd_workspace_bytes(linear_dims(rows=8, in_dim=65536)) == 0  # few rows: no scratch
    split = ms.gated_linear_fwd_workspace_bytes(linear_dims(rows=200, in_dim=65536))
    assert split >= 2 * 200 * 2 * 32 * 4  # both products of two shares at least
    assert ms.gated_linear_bwd_workspace_bytes(linear_dims()) >= 100 * 2 * 32 * 2
    for bad, _ in LINEAR_BAD + [(dict(out_dim=(1 << 19) + 8), 0)]:
        for query in (ms.gated_linear_fwd_workspace_bytes, ms.gated_linear_bwd_workspace_bytes):
            with pytest.raises(ms.MambaError):
                query(linear_dims(**bad))


def test_gated_refusals(lib):
    def fwd(d, x=FAKE, wg=FAKE, wu=FAKE, bg=None, bu=None, out=FAKE, pre=None):
        return lib.mamba_gated_linear_fwd(x, wg, wu, bg, bu, d and ctypes.byref(d), out, pre, None)

    def bwd(d, x=FAKE, wg=FAKE, wu=FAKE, pre=FAKE, dout=FAKE, dx=FAKE, dwg=FAKE, dwu=FAKE, dbg=FAKE, dbu=FAKE):
        return lib.mamba_gated_linear_bwd(x, wg, wu, pre, dout, d and ctypes.byref(d), dx, dwg, dwu, dbg, dbu, None)

    for call, needed in ((fwd, ("x", "wg", "wu", "out")), (bwd, ("x", "wg", "wu", "pre", "dout", "dwg", "dwu", "dbg", "dbu"))):
        assert call(None) == E.MAMBA_ERR_INVALID
        for miss in needed:  # (of a pair of outputs, one alone)
            assert call(linear_dims(), **{miss: None}) == E.MAMBA_ERR_INVALID, miss
        for bad, code in LINEAR_BAD + [(dict(out_dim=(1 << 19) + 8), E.MAMBA_ERR_UNSUPPORTED)]:
            assert call(linear_dims(**bad)) == code, bad
    assert bwd(linear_dims(), dx=None, dwg=None, dwu=None, dbg=None, dbu=None) == E.MAMBA_ERR_INVALID
    for call, odd in ((fwd, ("x", "wg", "wu", "out", "pre")), (bwd, ("x", "wg", "wu", "pre", "dout", "dx", "dwg", "dwu"))):
        for k in odd:
            assert call(linear_dims(), **{k: FAKE + 8}) == E.MAMBA_ERR_UNSUPPORTED, k
    for call, odd in ((fwd, ("bg", "bu")), (bwd, ("dbg", "dbu"))):
        for k in odd:
            assert call(linear_dims(), **{k: FAKE + 2}) == E.MAMBA_ERR_UNSUPPORTED, k
    assert fwd(linear_dims(rows=200, in_dim=65536)) == E.MAMBA_ERR_WORKSPACE
    need = ms.gated_linear_fwd_workspace_bytes(linear_dims(rows=200, in_dim=65536))
    assert fwd(linear_dims(rows=200, in_dim=65536, workspace=FAKE, workspace_bytes=need - 1)) == E.MAMBA_ERR_WORKSPACE
    assert bwd(linear_dims()) == E.MAMBA_ERR_WORKSPACE
    need = ms.gated_linear_bwd_workspace_bytes(linear_dims())
    assert bwd(linear_dims(workspace=FAKE, workspace_bytes=need - 1)) == E.MAMBA_ERR_WORKSPACE


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_gated_reference_gradients_against_differences(act):
    n = maker(9, "cpu")
    v = dict(x=n((5, 12)).double(), wg=n((7, 12)).double(), wu=n((7, 12)).double(), bg=n((7,)).double(), bu=n((7,)).double())
    dout = n((5, 7)).double()
    _, g, _, grads = gated_ref(**v, act=act, dout=dout)
    eps = 1e-6
    assert float(g.abs().min()) > 100 * eps  # no step crosses relu's kink
    for k, gk in (("x", "dx"), ("wg", "dw_gate"), ("wu", "dw_up"), ("bg", "db_gate"), ("bu", "db_up")):
        d = n(tuple(v[k].shape)).double()
        f = lambda s: float((gated_ref(**dict(v, **{k: v[k] + s * d}), act=act)[0] * dout).sum())  # noqa: E731
        num = (f(eps) - f(-eps)) / (2 * eps)
        want = float((grads[gk] * d).sum())
        assert abs(num - want) <= 1e-6 * max(1.0, abs(want)), (k, num, want)


def test_quant_sizes_and_refusals(lib):
    assert ms.linear_q8_workspace_bytes(linear_dims()) == 0
    assert ms.linear_q8_workspace_bytes(linear_dims(rows=8, in_dim=65536)) == 0
    need = ms.linear_q8_workspace_bytes(linear_dims(rows=200, in_dim=65536))
    assert need > 0

    def q8(d, x=FAKE, sx=FAKE, w=FAKE, sw=FAKE, b=None, res=None, out=FAKE):
        return lib.mamba_linear_q8(x, sx, w, sw, b, res, d and ctypes.byref(d), out, None)

    assert q8(None) == E.MAMBA_ERR_INVALID
    for miss in ("x", "sx", "w", "sw", "out"):
        assert q8(linear_dims(), **{miss: None}) == E.MAMBA_ERR_INVALID
    for bad, code in LINEAR_BAD + [(dict(in_dim=72), E.MAMBA_ERR_UNSUPPORTED)]:
        assert q8(linear_dims(**bad)) == code, bad
        with pytest.raises(ms.MambaError):
            ms.linear_q8_workspace_bytes(linear_dims(**bad))
    for odd in ("x", "w", "res", "out"):
        assert q8(linear_dims(), **{odd: FAKE + 8}) == E.MAMBA_ERR_UNSUPPORTED
    for odd in ("sx", "sw", "b"):
        assert q8(linear_dims(), **{odd: FAKE + 2}) == E.MAMBA_ERR_UNSUPPORTED
    assert q8(linear_dims(rows=200, in_dim=65536)) == E.MAMBA_ERR_WORKSPACE
    assert q8(linear_dims(rows=200, in_dim=65536, workspace=FAKE, workspace_bytes=need - 1)) == E.MAMBA_ERR_WORKSPACE

    def dims4(**kw):
        base = dict(rows=4, in_dim=64, out_dim=32, group=64, dtype=ms.DTYPE_BF16)
        base.update(kw)
        return ms.make_q4_dims(base.pop("rows"), base.pop("in_dim"), base.pop("out_dim"), base.pop("group"), base.pop("dtype"), **base)

    def q4(d, x=FAKE, w=FAKE, s=FAKE, z=None, b=None, res=None, out=FAKE):
        return lib.mamba_linear_q4(x, w, s, z, b, res, d and ctypes.byref(d), out, None)

    assert q4(None) == E.MAMBA_ERR_INVALID
    for miss in ("x", "w", "s", "out"):
        assert q4(dims4(), **{miss: None}) == E.MAMBA_ERR_INVALID
    for bad in (dict(rows=0), dict(in_dim=0), dict(out_dim=-8), dict(group=0), dict(group=-32), dict(dtype=2), dict(scale_dtype=2),
                dict(act=-1)):
        assert q4(dims4(**bad)) == E.MAMBA_ERR_INVALID, bad
    for bad in (dict(in_dim=48), dict(out_dim=20), dict(group=16), dict(group=96), dict(group=160), dict(in_dim=(1 << 20) + 32),
                dict(out_dim=(1 << 20) + 8), dict(rows=(1 << 18) + 1), dict(group=(1 << 20) + 128)):
        assert q4(dims4(**bad)) == E.MAMBA_ERR_UNSUPPORTED, bad
    for odd in ("x", "w", "res", "out"):
        assert q4(dims4(), **{odd: FAKE + 8}) == E.MAMBA_ERR_UNSUPPORTED
    assert q4(dims4(), s=FAKE + 1) == E.MAMBA_ERR_UNSUPPORTED
    assert q4(dims4(scale_dtype=ms.DTYPE_F32), s=FAKE + 2) == E.MAMBA_ERR_UNSUPPORTED
    assert q4(dims4(), b=FAKE + 2) == E.MAMBA_ERR_UNSUPPORTED

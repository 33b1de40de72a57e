"""Host-side checks of the operators around the scan (no GPU work): sizes,
refusals before any launch, and the float64 references' gradients against
differences."""
import ctypes
import os

import numpy as np
import pytest

import selective_state_space_mamba_amd as ms
from selective_state_space_mamba_amd import _binding as E

from layerutil import glr_grads, glr_ref

FAKE = 0x100000  # 16-byte aligned stand-in pointer: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ms.LIB_PATH):
        from selective_state_space_mamba_amd import build
        build.build(force=False)
    return ms.load_library()


def glr_dims(**kw):
    base = dict(batch=2, seqlen=100, dim=64, dtype=ms.DTYPE_BF16)
    base.update(kw)
    return ms.make_glr_dims(base.pop("batch"), base.pop("seqlen"), base.pop("dim"), base.pop("dtype"), **base)


def test_glr_sizes(lib):
    assert ms.glr_fwd_workspace_bytes(glr_dims()) == 0  # one tile: nothing to join
    assert ms.glr_fwd_workspace_bytes(glr_dims(seqlen=1000)) > 0
    assert ms.glr_fwd_workspace_bytes(glr_dims(seqlen=1000, batch=4096)) == 0  # enough rows: tiles walked in order
    assert ms.glr_bwd_workspace_bytes(glr_dims()) > 0
    assert ms.glr_saved_bytes(glr_dims()) == 2 * 2 * 64 * 4
    assert ms.glr_saved_bytes(glr_dims(seqlen=128)) == 2 * 2 * 64 * 4
    assert ms.glr_saved_bytes(glr_dims(seqlen=129)) == 2 * 3 * 64 * 4
    for bad in (dict(batch=0), dict(seqlen=0), dict(dim=-4), dict(dim=6), dict(dtype=4), dict(input_rule=3),
                dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(dim=1 << 22),
                dict(seqlen=(1 << 31) - 64), dict(batch=1 << 24, seqlen=1 << 20)):
        for query in (ms.glr_fwd_workspace_bytes, ms.glr_bwd_workspace_bytes, ms.glr_saved_bytes):
            with pytest.raises(ms.MambaError):
                query(glr_dims(**bad))


def test_glr_refusals(lib):
    def fwd(d, **kw):
        p = dict(x=FAKE, r=FAKE, i=None, z=None, lam=None, out=FAKE, last=None, saved=None, n=0)
        p.update(kw)
        return lib.mamba_glr_fwd(p["x"], p["r"], p["i"], p["z"], p["lam"], ctypes.byref(d), p["out"], p["last"],
                                 p["saved"], p["n"], None)

    for miss in ("x", "r", "out"):
        assert fwd(glr_dims(), **{miss: None}) == E.MAMBA_ERR_INVALID
    assert fwd(glr_dims(batch=0)) == E.MAMBA_ERR_INVALID
    assert fwd(glr_dims(dim=66)) == E.MAMBA_ERR_UNSUPPORTED
    for odd in ("x", "r", "i", "z", "lam", "out", "last", "saved"):
        assert fwd(glr_dims(), **{odd: FAKE + 8, "n": 1 << 30}) == E.MAMBA_ERR_UNSUPPORTED
    assert fwd(glr_dims(), saved=FAKE, n=2 * 2 * 64 * 4 - 1) == E.MAMBA_ERR_WORKSPACE
    assert fwd(glr_dims(seqlen=1000)) == E.MAMBA_ERR_WORKSPACE
    need = ms.glr_fwd_workspace_bytes(glr_dims(seqlen=1000))
    assert fwd(glr_dims(seqlen=1000, workspace=FAKE, workspace_bytes=need - 1)) == E.MAMBA_ERR_WORKSPACE

    def bwd(d, **kw):
        p = dict(x=FAKE, r=FAKE, i=None, z=None, lam=None, dout=FAKE, dx=FAKE, dr=FAKE, di=None, dz=None, dlam=None,
                 saved=None, n=0)
        p.update(kw)
        return lib.mamba_glr_bwd(p["x"], p["r"], p["i"], p["z"], p["lam"], p["dout"], None, ctypes.byref(d), p["dx"],
                                 p["dr"], p["di"], p["dz"], p["dlam"], None, p["saved"], p["n"], None)

    for miss in ("x", "r", "dout", "dx", "dr"):
        assert bwd(glr_dims(), **{miss: None}) == E.MAMBA_ERR_INVALID
    assert bwd(glr_dims(), i=FAKE) == E.MAMBA_ERR_INVALID  # i's gradient has nowhere to go
    assert bwd(glr_dims(), z=FAKE) == E.MAMBA_ERR_INVALID
    assert bwd(glr_dims(), dr=FAKE + 4) == E.MAMBA_ERR_UNSUPPORTED
    assert bwd(glr_dims()) == E.MAMBA_ERR_WORKSPACE
    need = ms.glr_bwd_workspace_bytes(glr_dims())
    assert bwd(glr_dims(workspace=FAKE, workspace_bytes=need - 1)) == E.MAMBA_ERR_WORKSPACE
    assert bwd(glr_dims(workspace=FAKE, workspace_bytes=need), saved=FAKE, n=16) == E.MAMBA_ERR_WORKSPACE

    def step(d, **kw):
        p = dict(state=FAKE, x=FAKE, r=FAKE, out=FAKE)
        p.update(kw)
        return lib.mamba_glr_step(p["state"], p["x"], p["r"], None, None, None, ctypes.byref(d), p["out"], None)

    for miss in ("state", "x", "r", "out"):
        assert step(glr_dims(), **{miss: None}) == E.MAMBA_ERR_INVALID
    assert step(glr_dims(dim=0)) == E.MAMBA_ERR_INVALID
    assert step(glr_dims(), state=FAKE + 4) == E.MAMBA_ERR_UNSUPPORTED
    assert lib.mamba_glr_step(FAKE, FAKE, FAKE, None, None, None, None, FAKE, None) == E.MAMBA_ERR_INVALID


@pytest.mark.parametrize("rule", ["sqrt", "lerp", "unit"])
@pytest.mark.parametrize("with_lam", [True, False])
@pytest.mark.parametrize("reverse", [True, False])
def test_glr_reference_gradients_against_differences(rule, with_lam, reverse):
    """Central differences in float64: relative error near eps² = 1e-10 plus 1e-16/eps; 1e-7 is asked."""
    r = np.random.Generator(np.random.PCG64(9))
    B, L, D = 2, 13, 3
    v = {k: r.standard_normal((B, L, D)) for k in ("x", "r", "i", "z")}
    v["lam"] = r.uniform(-4, 0, D) if with_lam else None
    v["init"] = r.standard_normal((B, D))
    dout, dlast = r.standard_normal((B, L, D)), r.standard_normal((B, D))
    reset = (r.uniform(size=(B, L)) < 0.2).astype(np.uint8)

    def loss(u):
        out, last, _, _ = glr_ref(u["x"], u["r"], u["i"], u["z"], u["lam"], rule=rule, reverse=reverse,
                                  init=u["init"], reset=reset)
        return (out * dout).sum() + (last * dlast).sum()

    g = glr_grads(v["x"], v["r"], v["i"], v["z"], v["lam"], dout, dlast, rule=rule, reverse=reverse, init=v["init"],
                  reset=reset)
    for k in ("x", "r", "i", "z", "lam", "init"):
        if v[k] is None:
            continue
        d = r.standard_normal(v[k].shape)
        eps = 1e-5
        num = (loss(dict(v, **{k: v[k] + eps * d})) - loss(dict(v, **{k: v[k] - eps * d}))) / (2 * eps)
        want = (g["d" + k] * d).sum()
        assert abs(num - want) <= 1e-7 * max(1.0, abs(want)), (k, num, want)


def norm_dims(**kw):
    base = dict(batch=2, seqlen=100, dim=64, groups=8, dtype=ms.DTYPE_BF16)
    base.update(kw)
    return ms.make_norm_dims(base.pop("batch"), base.pop("seqlen"), base.pop("dim"), base.pop("groups"),
                             base.pop("dtype"), **base)


def test_norm_sizes(lib):
    assert ms.group_norm_fwd_workspace_bytes(norm_dims(seqlen=1)) == 0
    assert ms.group_norm_fwd_workspace_bytes(norm_dims(seqlen=100000)) > 0
    assert ms.group_norm_bwd_workspace_bytes(norm_dims(seqlen=1)) >= 2 * 64 * 8
    for bad in (dict(batch=0), dict(seqlen=0), dict(dim=0), dict(groups=0), dict(groups=7), dict(dim=60, groups=4),
                dict(dim=8200, groups=1), dict(act=4), dict(act=-1), dict(dtype=3), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(seqlen=1 << 31), dict(batch=1 << 31)):
        for query in (ms.group_norm_fwd_workspace_bytes, ms.group_norm_bwd_workspace_bytes):
            with pytest.raises(ms.MambaError):
                query(norm_dims(**bad))


def test_norm_refusals(lib):
    def fwd(d, x=FAKE, w=None, b=None, out=FAKE, mean=None):
        return lib.mamba_group_norm_fwd(x, w, b, ctypes.byref(d), out, mean, None, None)

    assert fwd(norm_dims(), x=None) == E.MAMBA_ERR_INVALID
    assert fwd(norm_dims(), out=None) == E.MAMBA_ERR_INVALID
    assert fwd(norm_dims(groups=7)) == E.MAMBA_ERR_INVALID
    assert fwd(norm_dims(dim=60, groups=4)) == E.MAMBA_ERR_UNSUPPORTED
    assert fwd(norm_dims(), x=FAKE + 8) == E.MAMBA_ERR_UNSUPPORTED
    assert fwd(norm_dims(), out=FAKE + 2) == E.MAMBA_ERR_UNSUPPORTED
    assert fwd(norm_dims(), w=FAKE + 2) == E.MAMBA_ERR_UNSUPPORTED
    assert fwd(norm_dims(), mean=FAKE + 1) == E.MAMBA_ERR_UNSUPPORTED
    assert fwd(norm_dims(seqlen=100000)) == E.MAMBA_ERR_WORKSPACE
    need = ms.group_norm_fwd_workspace_bytes(norm_dims(seqlen=100000))
    assert fwd(norm_dims(seqlen=100000, workspace=FAKE, workspace_bytes=need - 1)) == E.MAMBA_ERR_WORKSPACE
    assert lib.mamba_group_norm_fwd(FAKE, None, None, None, FAKE, None, None, None) == E.MAMBA_ERR_INVALID

    def bwd(d, **kw):
        p = dict(x=FAKE, dout=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE)
        p.update(kw)
        return lib.mamba_group_norm_bwd(p["x"], None, None, p["dout"], p["mean"], p["rstd"], ctypes.byref(d), p["dx"],
                                        None, None, None)

    for miss in ("x", "dout", "mean", "rstd", "dx"):
        assert bwd(norm_dims(), **{miss: None}) == E.MAMBA_ERR_INVALID
    for odd in ("x", "dout", "dx"):
        assert bwd(norm_dims(), **{odd: FAKE + 8}) == E.MAMBA_ERR_UNSUPPORTED
    assert bwd(norm_dims()) == E.MAMBA_ERR_WORKSPACE


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_norm_reference_gradients_against_differences(act):
    from layerutil import norm_ref
    r = np.random.Generator(np.random.PCG64(4))
    B, L, D, G = 2, 5, 12, 3
    v = dict(x=r.standard_normal((B, L, D)), w=r.standard_normal(D), b=r.standard_normal(D))
    dout = r.standard_normal((B, L, D))
    g = norm_ref(v["x"], G, v["w"], v["b"], act, 1e-5, dout)[3]
    for k, gk in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
        d = r.standard_normal(v[k].shape)
        eps = 1e-6 if act == "relu" else 1e-5
        f = lambda s: (norm_ref(**{**{"G": G, "act": act, "eps": 1e-5}, **v, k: v[k] + s * d})[0] * dout).sum()  # noqa: E731
        num = (f(eps) - f(-eps)) / (2 * eps)
        want = (g[gk] * d).sum()
        assert abs(num - want) <= 1e-6 * max(1.0, abs(want)), (k, num, want)


def linear_dims(**kw):
    base = dict(rows=100, in_dim=64, out_dim=32, dtype=ms.DTYPE_BF16)
    base.update(kw)
    return ms.make_linear_dims(base.pop("rows"), base.pop("in_dim"), base.pop("out_dim"), base.pop("dtype"), **base)


def test_linear_sizes(lib):
    assert ms.linear_fwd_workspace_bytes(linear_dims()) == 0
    assert ms.linear_fwd_workspace_bytes(linear_dims(rows=8, in_dim=65536)) == 0  # few rows: no scratch
    assert ms.linear_fwd_workspace_bytes(linear_dims(rows=200, in_dim=65536)) > 0  # split contraction
    assert ms.linear_bwd_workspace_bytes(linear_dims(act=ms.ACT_SILU)) > 100 * 32 * 2
    for bad in (dict(rows=0), dict(in_dim=0), dict(out_dim=-8), dict(in_dim=12), dict(out_dim=20), dict(dtype=2),
                dict(act=4), dict(in_dim=(1 << 20) + 8), dict(out_dim=(1 << 20) + 8), dict(rows=(1 << 29) + 1)):
        for query in (ms.linear_fwd_workspace_bytes, ms.linear_bwd_workspace_bytes):
            with pytest.raises(ms.MambaError):
                query(linear_dims(**bad))


def test_linear_refusals(lib):
    def fwd(d, x=FAKE, w=FAKE, b=None, res=None, out=FAKE, pre=None):
        return lib.mamba_linear_fwd(x, w, b, res, ctypes.byref(d), out, pre, None)

    for miss in ("x", "w", "out"):
        assert fwd(linear_dims(), **{miss: None}) == E.MAMBA_ERR_INVALID
    assert fwd(linear_dims(act=-1)) == E.MAMBA_ERR_INVALID
    assert fwd(linear_dims(in_dim=4)) == E.MAMBA_ERR_UNSUPPORTED
    for odd in ("x", "w", "res", "out", "pre"):
        assert fwd(linear_dims(), **{odd: FAKE + 8}) == E.MAMBA_ERR_UNSUPPORTED
    assert fwd(linear_dims(), b=FAKE + 2) == E.MAMBA_ERR_UNSUPPORTED
    assert fwd(linear_dims(rows=200, in_dim=65536)) == E.MAMBA_ERR_WORKSPACE
    assert lib.mamba_linear_fwd(FAKE, FAKE, None, None, None, FAKE, None, None) == E.MAMBA_ERR_INVALID

    def bwd(d, **kw):
        p = dict(x=FAKE, w=FAKE, pre=None, dout=FAKE, dx=FAKE, dw=FAKE, db=FAKE)
        p.update(kw)
        return lib.mamba_linear_bwd(p["x"], p["w"], p["pre"], p["dout"], ctypes.byref(d), p["dx"], p["dw"], p["db"],
                                    None)

    for miss in ("x", "w", "dout"):
        assert bwd(linear_dims(), **{miss: None}) == E.MAMBA_ERR_INVALID
    assert bwd(linear_dims(), dx=None, dw=None, db=None) == E.MAMBA_ERR_INVALID
    assert bwd(linear_dims(act=ms.ACT_GELU)) == E.MAMBA_ERR_INVALID  # no pre
    assert bwd(linear_dims(), dw=FAKE + 8) == E.MAMBA_ERR_UNSUPPORTED
    assert bwd(linear_dims()) == E.MAMBA_ERR_WORKSPACE
    need = ms.linear_bwd_workspace_bytes(linear_dims())
    assert bwd(linear_dims(workspace=FAKE, workspace_bytes=need - 1)) == E.MAMBA_ERR_WORKSPACE


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_linear_reference_gradients_against_differences(act):
    from layerutil import linear_ref
    r = np.random.Generator(np.random.PCG64(14))
    v = dict(x=r.standard_normal((5, 12)), w=r.standard_normal((7, 12)), b=r.standard_normal(7))
    dout = r.standard_normal((5, 7))
    pre, g = linear_ref(v["x"], v["w"], v["b"], None, act, dout)[1:]
    eps = 1e-6
    assert np.abs(pre).min() > 100 * eps  # no step crosses relu's kink
    for k, gk in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
        d = r.standard_normal(v[k].shape)
        f = lambda s: (linear_ref(**{"res": None, "act": act, **v, k: v[k] + s * d})[0] * dout).sum()  # noqa: E731
        num = (f(eps) - f(-eps)) / (2 * eps)
        want = (g[gk] * d).sum()
        assert abs(num - want) <= 1e-6 * max(1.0, abs(want)), (k, num, want)

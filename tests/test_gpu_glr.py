"""GPU parity of the gated linear recurrence (mamba_glr_*, through the C ABI)
with its plain float64 form (layerutil), for every input rule, with and without
lam, gates, resets, an initial state and the reversed order; lengths from one
token past several tiles (64 and 128 positions) and channel counts that end
inside a 64-channel block.

Tolerances, written before the first run.  float32: a decay is rounded to
2^-24 and a state remembers up to 1/(1 - a) = 1000 positions here, so its
relative error stays below 1000·2^-24 = 6e-5 and, the roundings being
independent, near sqrt(1000)·2^-24 = 2e-6 in the L2 norm; the project's float32
bar of 2e-4 (normwise) covers the first and 2e-5 is taken for the second.
bfloat16: the output rounding, 2^-9 of a value, against the project's 1e-2
(normwise) and 3e-3 (L2).  float32 sums beside bfloat16 data (states, dlam,
dinit) are held to the float32 bar."""
import numpy as np
import pytest

import selective_state_space_mamba_amd as ms

from layerutil import from_dev, glr_grads, glr_ref, rounded, to_dev
from scanutil import errors, torch

pytestmark = pytest.mark.gpu

RULES = {"sqrt": ms.GLR_SQRT, "lerp": ms.GLR_LERP, "unit": ms.GLR_UNIT}
TOL = {"f32": (2e-4, 2e-5), "bf16": (1e-2, 3e-3)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield


def close(name, got, want, dtype):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, name
    assert np.all(np.isfinite(got)), name
    emax, el2 = errors(got, want)
    print("%s: max %.2e l2 %.2e" % (name, emax, el2), flush=True)
    assert emax <= TOL[dtype][0] and el2 <= TOL[dtype][1], (name, emax, el2)


def make(B, L, D, dtype, seed, *, lam=True, i=True, z=True, reset=0.0, init=True):
    r = np.random.Generator(np.random.PCG64([seed, 77]))
    dev, ref = {}, {}
    for k, on in (("x", True), ("r", True), ("i", i), ("z", z), ("dout", True)):
        dev[k], ref[k] = (None, None) if not on else rounded(r.standard_normal((B, L, D)), dtype)
        dev[k] = to_dev(dev[k])
    for k, on, shape in (("init", init, (B, D)), ("dlast", init, (B, D))):
        v = r.standard_normal(shape).astype(np.float32) if on else None
        dev[k], ref[k] = to_dev(v), None if v is None else v.astype(np.float64)
    v = None
    if lam:  # decays between 0.9 and 0.999 at an open gate
        v = np.log(np.expm1(-np.log(r.uniform(0.9, 0.999, D)) / 8.0)).astype(np.float32)
    dev["lam"], ref["lam"] = to_dev(v), None if v is None else v.astype(np.float64)
    m = (r.uniform(size=(B, L)) < reset).astype(np.uint8) if reset else None
    dev["reset"], ref["reset"] = to_dev(m), m
    return dev, ref


def kwargs(v, rule, reverse, ref):
    return dict(init=v["init"], reset=v["reset"], rule=rule, reverse=reverse) if ref else dict(
        initial_state=v["init"], reset=v["reset"], input_rule=RULES[rule], reverse=reverse)


def args(v):
    return v["x"], v["r"], v["i"], v["z"], v["lam"]


CASES = [
    # B, L, D, dtype, rule, reverse, options
    (2, 1, 64, "bf16", "sqrt", False, {}),
    (1, 1, 4, "f32", "lerp", True, dict(init=False)),
    (3, 63, 68, "f32", "sqrt", False, {}),
    (2, 64, 72, "bf16", "lerp", False, dict(i=False)),
    (2, 65, 8, "f32", "unit", True, dict(z=False)),
    (1, 129, 200, "bf16", "sqrt", True, {}),
    (2, 300, 136, "f32", "sqrt", False, dict(reset=0.03)),
    (2, 300, 132, "bf16", "lerp", True, dict(reset=0.03, lam=False)),
    (1, 1025, 68, "f32", "sqrt", False, dict(lam=False, z=False, i=False, init=False)),
    (1, 2309, 260, "f32", "lerp", False, dict(reset=0.003)),
    (1, 4133, 64, "bf16", "unit", False, dict(init=False)),
    (2, 5000, 12, "f32", "sqrt", True, dict(reset=0.002)),
    # enough rows for one workgroup to walk all its tiles
    (40, 200, 1664, "bf16", "sqrt", False, {}),
    (33, 131, 2052, "f32", "lerp", True, dict(reset=0.02)),
    (64, 140, 2080, "f32", "unit", False, dict(reset=0.02)),
    (64, 70, 2052, "bf16", "sqrt", True, dict(lam=False)),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d-L%d-D%d-%s-%s-rev%d" % c[:6])
def test_forward_and_gradients(case):
    B, L, D, dtype, rule, reverse, opt = case
    print("[gpu case] glr", case, flush=True)
    dev, ref = make(B, L, D, dtype, L + D, **opt)
    kw = kwargs(dev, rule, reverse, False)
    out, last = ms.glr_fwd(*args(dev), **kw)
    torch().cuda.synchronize()
    want, want_last, _, _ = glr_ref(*args(ref), **kwargs(ref, rule, reverse, True))
    close("out", from_dev(out), want, dtype)
    close("last_state", from_dev(last), want_last, "f32")
    out2, last2, saved = ms.glr_fwd_save(*args(dev), **kw)
    assert torch().equal(out, out2) and torch().equal(last, last2)
    g = ms.glr_bwd(*args(dev), dout=dev["dout"], dlast=dev["dlast"], saved=saved, **kw)
    again = ms.glr_bwd(*args(dev), dout=dev["dout"], dlast=dev["dlast"], **kw)
    torch().cuda.synchronize()
    wg = glr_grads(*args(ref), ref["dout"], ref["dlast"], **kwargs(ref, rule, reverse, True))
    for k in ("dx", "dr", "di", "dz", "dlam", "dinit"):
        assert (g[k] is None) == (wg[k] is None), k
        if g[k] is not None:
            close(k, from_dev(g[k]), wg[k], "f32" if k in ("dlam", "dinit") else dtype)
            assert torch().equal(g[k], again[k]), k  # recomputed states: the same bits


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_chain_gives_the_same_bits_every_time(dtype):
    """Few rows, many tiles: the tiles run at once and join through memory."""
    dev, _ = make(1, 20000, 192, dtype, 5, reset=0.0005)
    kw = kwargs(dev, "sqrt", False, False)
    first = None
    for _ in range(4):
        out, last, saved = ms.glr_fwd_save(*args(dev), **kw)
        g = ms.glr_bwd(*args(dev), dout=dev["dout"], saved=saved, **kw)
        got = [out, last] + [g[k] for k in sorted(g)]
        if first is not None:
            assert all(torch().equal(a, b) for a, b in zip(first, got))
        first = got


@pytest.mark.parametrize("rule", sorted(RULES))
@pytest.mark.parametrize("lam", [True, False])
def test_steps_continue_the_scan(rule, lam):
    B, L, D, n = 3, 70, 76, 9
    for dtype in ("f32", "bf16"):
        dev, ref = make(B, L + n, D, dtype, 11, lam=lam)
        cut = {k: (v[:, :L].contiguous() if v is not None and v.dim() == 3 else v) for k, v in dev.items()}
        _, state = ms.glr_fwd(*args(cut), initial_state=dev["init"], input_rule=RULES[rule])
        outs = []
        for t in range(L, L + n):
            tok = [None if v is None else v[:, t].contiguous() for v in args(dev)[:4]]
            outs.append(ms.glr_step(state, *tok, dev["lam"], input_rule=RULES[rule]))
        torch().cuda.synchronize()
        want, want_last, _, _ = glr_ref(*args(ref), init=ref["init"], rule=rule)
        close("steps", np.stack([from_dev(o) for o in outs], 1), want[:, L:], dtype)
        close("state", from_dev(state), want_last, "f32")


def test_decays_near_one_keep_their_input_factor():
    """E down to 1e-7: 1 - a and sqrt(1 - a²) must not be lost to the subtraction."""
    B, L, D = 1, 3, 64
    r = np.linspace(-17.0, -1.0, B * L * D).reshape(B, L, D).astype(np.float32)
    x = np.ones((B, L, D), np.float32)
    lam = np.full(D, -4.0, np.float32)
    for rule in ("sqrt", "lerp"):
        out, _ = ms.glr_fwd(to_dev(x), to_dev(r), lam=to_dev(lam), input_rule=RULES[rule])
        want = glr_ref(x.astype(np.float64), r.astype(np.float64), None, None, lam.astype(np.float64), rule=rule)[0]
        rel = np.abs(from_dev(out) - want) / want
        assert rel.max() < 1e-5, (rule, rel.max())  # ulps of two exponentials and a square root, over three positions


def test_saturated_gates():
    """Gates far outside their usual range: decays of 0 and 1, closed and open input gates."""
    B, L, D = 2, 150, 64
    r = np.random.Generator(np.random.PCG64(3))
    vals = np.array([-200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0], np.float32)
    raw = {k: vals[r.integers(0, 7, (B, L, D))] for k in ("r", "i", "z")}
    raw["x"] = r.standard_normal((B, L, D)).astype(np.float32)
    dout = r.standard_normal((B, L, D)).astype(np.float32)
    lam = vals[r.integers(0, 5, D)]
    f8 = {k: v.astype(np.float64) for k, v in raw.items()}
    for rule in RULES:
        for lm in (lam, None):
            a = [to_dev(raw[k]) for k in "xriz"] + [to_dev(lm)]
            b = [f8[k] for k in "xriz"] + [None if lm is None else lm.astype(np.float64)]
            out, last = ms.glr_fwd(*a, input_rule=RULES[rule])
            g = ms.glr_bwd(*a, dout=to_dev(dout), input_rule=RULES[rule])
            with np.errstate(all="ignore"):
                want, want_last, _, _ = glr_ref(*b, rule=rule)
                wg = glr_grads(*b, dout.astype(np.float64), rule=rule)
            close("out %s" % rule, from_dev(out), want, "f32")
            close("last %s" % rule, from_dev(last), want_last, "f32")
            for k, v in g.items():
                if v is not None:
                    close("%s %s" % (k, rule), from_dev(v), wg[k], "f32")


@pytest.mark.parametrize("reverse", [False, True])
def test_resets_stop_nan_and_infinity(reverse):
    """A document that ends in NaN and infinities leaves the next one, and the gradients of the ones around it, alone."""
    B, L, D = 1, 700, 64
    for dtype in ("f32", "bf16"):
        dev, ref = make(B, L, D, dtype, 21)
        lo, hi = 200, 410  # the bad document
        starts = [lo, hi] if not reverse else [hi - 1, lo - 1]
        reset = np.zeros((B, L), np.uint8)
        reset[:, starts] = 1
        bad = {k: (v.clone() if v is not None else None) for k, v in dev.items()}
        bad["x"][:, lo:hi] = float("nan")
        bad["r"][:, lo + 3:hi:2] = float("nan")
        bad["x"][:, lo + 5:hi:3] = float("inf")
        kw = dict(input_rule=ms.GLR_SQRT, reverse=reverse, reset=to_dev(reset), initial_state=dev["init"])
        out, last, saved = ms.glr_fwd_save(*args(bad), **kw)
        g = ms.glr_bwd(*args(bad), dout=dev["dout"], saved=saved, **kw)
        good = np.r_[0:lo, hi:L]
        rkw = dict(rule="sqrt", reverse=reverse, reset=reset, init=ref["init"])
        want, want_last, _, _ = glr_ref(*args(ref), **rkw)
        wg = glr_grads(*args(ref), ref["dout"], **rkw)
        close("out", from_dev(out)[:, good], want[:, good], dtype)
        close("last", from_dev(last), want_last, "f32")
        for k in ("dx", "dr", "di", "dz"):
            close(k, from_dev(g[k])[:, good], wg[k][:, good], dtype)
        close("dinit", from_dev(g["dinit"]), wg["dinit"], "f32")


def test_gradients_against_differences():
    """Central differences of the kernel's own forward along random directions.  The forward's float32 rounding
    (relative 2e-6 of a sum of N terms, near 2e-6·sqrt(N) here) over a step of 2e-2 leaves about 1e-3 of the
    derivative, the step's second order about 1e-3 more; 1e-2 is asked."""
    B, L, D = 1, 90, 64
    for rule in RULES:
        dev, _ = make(B, L, D, "f32", 31, reset=0.02)
        kw = dict(input_rule=RULES[rule], reset=dev["reset"])

        def loss(v):
            out, last = ms.glr_fwd(*args(v), initial_state=v["init"], **kw)
            return float((out.double() * dev["dout"].double()).sum() + (last.double() * dev["dlast"].double()).sum())

        g = ms.glr_bwd(*args(dev), dout=dev["dout"], dlast=dev["dlast"], initial_state=dev["init"], **kw)
        for k, gk in (("x", "dx"), ("r", "dr"), ("i", "di"), ("z", "dz"), ("lam", "dlam"), ("init", "dinit")):
            d = torch().sign(g[gk])  # a direction that adds every component up
            eps = 1e-2
            up, down = dict(dev), dict(dev)
            up[k], down[k] = dev[k] + eps * d, dev[k] - eps * d
            num = (loss(up) - loss(down)) / (2 * eps)
            want = float((g[gk].double() * d.double()).sum())
            assert abs(num - want) <= 1e-2 * abs(want), (rule, k, num, want)


def test_other_stream_and_graph():
    t = torch()
    dev, _ = make(1, 3000, 128, "bf16", 41)
    kw = kwargs(dev, "sqrt", False, False)
    want, want_last = ms.glr_fwd(*args(dev), **kw)
    wg = ms.glr_bwd(*args(dev), dout=dev["dout"], **kw)
    t.cuda.synchronize()
    s = t.cuda.Stream()
    out, last = ms.glr_fwd(*args(dev), stream=s, **kw)
    g = ms.glr_bwd(*args(dev), dout=dev["dout"], stream=s, **kw)
    s.synchronize()
    assert t.equal(out, want) and t.equal(last, want_last)
    assert all(t.equal(g[k], wg[k]) for k in g)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        out, last, saved = ms.glr_fwd_save(*args(dev), **kw)
        g = ms.glr_bwd(*args(dev), dout=dev["dout"], saved=saved, **kw)
    for _ in range(3):
        for v in [out, last] + list(g.values()):
            v.zero_()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(out, want) and t.equal(last, want_last)
        assert all(t.equal(g[k], wg[k]) for k in g)
        junk = t.randn(1 << 20, device="cuda:0").sum().item()
        assert junk == junk


def test_binding_refusals():
    t = torch()
    x = t.zeros(2, 8, 64, device="cuda:0")
    with pytest.raises(ValueError):
        ms.glr_fwd(x, x[:, :4].contiguous())
    with pytest.raises(ValueError):
        ms.glr_fwd(x, x.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(TypeError):
        ms.glr_fwd(x, x.bfloat16())
    with pytest.raises(TypeError):
        ms.glr_fwd(x.half(), x.half())
    with pytest.raises(TypeError):
        ms.glr_fwd(x, x, reset=t.zeros(2, 8, device="cuda:0"))
    with pytest.raises(ms.MambaError):
        ms.glr_fwd(x[:, :, :6].contiguous(), x[:, :, :6].contiguous())
    with pytest.raises(ms.MambaError):
        ms.glr_fwd(x, x, scale=float("nan"))

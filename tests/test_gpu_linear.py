"""GPU parity of the matrix product with bias, activation and residual
(mamba_linear_*, through the C ABI) with its plain float64 form: one row, the
sizes on both sides of the few-rows kernel's limits, sizes that end inside every
tile and stage, split contractions, each activation, and each gradient alone.

Tolerances, written before the first run.  A float32 sum of K products errs by
about sqrt(K)·2^-24 of its scale, 4e-6 at K = 4096: 2e-4 (normwise) and 2e-5
(L2).  bfloat16 outputs carry one rounding (L2 2^-9/sqrt(3) = 1.1e-3): 1e-2 and
3e-3; gradients behind an activation one more (of dout·act'(pre)): 4e-3.  pre and
dbias are float32 sums throughout."""
import numpy as np
import pytest

import selective_state_space_mamba_amd as ms

from layerutil import ACTS, from_dev, linear_ref, rounded, to_dev
from scanutil import errors, torch

pytestmark = pytest.mark.gpu
TOL = {"f32": (2e-4, 2e-5), "bf16": (1e-2, 3e-3), "bf16 act": (2e-2, 4e-3)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield


def close(name, got, want, kind):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, name
    assert np.all(np.isfinite(got)), name
    emax, el2 = errors(got, want)
    print("%s: max %.2e l2 %.2e" % (name, emax, el2), flush=True)
    assert emax <= TOL[kind][0] and el2 <= TOL[kind][1], (name, emax, el2)


def make(M, K, N, dtype, seed, bias=True, res=True):
    r = np.random.Generator(np.random.PCG64([seed, 6]))
    v = dict(x=rounded(r.standard_normal((M, K)), dtype), w=rounded(r.standard_normal((N, K)) / np.sqrt(K), dtype),
             dout=rounded(r.standard_normal((M, N)), dtype))
    v["res"] = rounded(r.standard_normal((M, N)), dtype) if res else (None, None)
    b = (0.2 * r.standard_normal(N)).astype(np.float32)
    v["b"] = (b, b.astype(np.float64)) if bias else (None, None)
    return {k: to_dev(a) for k, (a, _) in v.items()}, {k: f for k, (_, f) in v.items()}


CASES = [
    # M, K, N, dtype, act, bias, residual
    (1, 8, 8, "f32", "none", True, True),
    (1, 8, 8, "bf16", "silu", True, False),
    (1, 1536, 768, "bf16", "none", True, True),
    (8, 1000, 24, "f32", "gelu", False, True),
    (15, 72, 200, "bf16", "relu", True, True),
    (17, 4096, 40, "bf16", "silu", True, False),
    (33, 264, 1032, "f32", "silu", True, True),
    (64, 40, 136, "bf16", "gelu", True, True),
    (65, 40, 136, "bf16", "gelu", True, True),
    (127, 8, 8, "bf16", "none", False, False),
    (129, 72, 136, "f32", "relu", True, True),
    (128, 128, 128, "bf16", "none", False, False),
    (200, 2056, 264, "bf16", "silu", True, True),
    (200, 2056, 264, "f32", "gelu", True, True),
    (1000, 200, 96, "f32", "none", True, False),
    (1500, 768, 1544, "bf16", "silu", True, False),
    (5003, 520, 256, "bf16", "gelu", True, True),
    (2100, 264, 1048, "bf16", "relu", False, True),
    # few rows whose contraction ends inside a turn; float32 tiles with half their columns or rows, or a quarter
    (40, 2008, 48, "bf16", "relu", True, True),
    (64, 1048, 72, "f32", "relu", True, True),
    (300, 96, 56, "f32", "silu", True, True),
    (333, 264, 152, "f32", "none", True, False),
    (3000, 40, 24, "f32", "gelu", True, True),
    # enough tiles for the large ones, the last of them partly empty, in each of the three products
    (16300, 328, 1528, "bf16", "silu", True, True),
    (8200, 1000, 2056, "bf16", "none", True, True),
    (2050, 2056, 2056, "bf16", "gelu", True, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%dx%d-%s-%s-b%d-r%d" % c)
def test_forward_and_gradients(case):
    M, K, N, dtype, act, bias, res = case
    print("[gpu case] linear", case, flush=True)
    dev, ref = make(M, K, N, dtype, M + K + N, bias, res)
    out, pre = ms.linear_fwd(dev["x"], dev["w"], dev["b"], dev["res"], act=ACTS[act], want_pre=act != "none")
    g = ms.linear_bwd(dev["x"], dev["w"], dout=dev["dout"], pre=pre, act=ACTS[act])
    torch().cuda.synchronize()
    want, wpre, wg = linear_ref(ref["x"], ref["w"], ref["b"], ref["res"], act, ref["dout"])
    close("out", from_dev(out), want, dtype)
    if act != "none":
        close("pre", from_dev(pre), wpre, "f32")
    kind = dtype if dtype == "f32" or act == "none" else "bf16 act"
    close("dx", from_dev(g["dx"]), wg["dx"], kind)
    close("dweight", from_dev(g["dweight"]), wg["dweight"], kind)
    close("dbias", from_dev(g["dbias"]), wg["dbias"], "f32")
    again = ms.linear_bwd(dev["x"], dev["w"], dout=dev["dout"], pre=pre, act=ACTS[act])
    assert all(torch().equal(g[k], again[k]) for k in g)
    for k in g:  # each gradient by itself
        one = ms.linear_bwd(dev["x"], dev["w"], dout=dev["dout"], pre=pre, act=ACTS[act],
                            **{"want_" + j: j == k for j in g})
        assert torch().equal(one[k], g[k]) and all(one[j] is None for j in g if j != k)


def test_exact_products():
    """Small whole numbers: every sum is exact in float32, so the tiles' layout shows without a tolerance."""
    r = np.random.Generator(np.random.PCG64(1))
    for dtype in ("f32", "bf16"):
        for M, K, N in ((5, 48, 32), (130, 88, 72), (300, 1032, 136)):
            x, w = r.integers(-2, 3, (M, K)), r.integers(-1, 2, (N, K))
            dout = r.integers(-1, 2, (M, N))
            a = [to_dev(rounded(v, dtype)[0]) for v in (x, w, dout)]
            out, _ = ms.linear_fwd(a[0], a[1])
            g = ms.linear_bwd(a[0], a[1], dout=a[2])
            for got, want in ((out, x @ w.T), (g["dx"], dout @ w), (g["dweight"], dout.T @ x)):
                assert np.array_equal(from_dev(got), rounded(want, dtype)[1])
            assert np.array_equal(from_dev(g["dbias"]), dout.sum(0))


@pytest.mark.parametrize("M", [3, 700])
def test_residual_in_place_and_leading_axes(M):
    dev, ref = make(M, 64, 96, "bf16", 9)
    want, _ = ms.linear_fwd(dev["x"], dev["w"], dev["b"], dev["res"], act=ms.ACT_GELU)
    buf = dev["res"].clone()
    got, _ = ms.linear_fwd(dev["x"], dev["w"], dev["b"], buf, act=ms.ACT_GELU, out=buf)
    assert got is buf and torch().equal(got, want)
    x3 = dev["x"][None]
    got, _ = ms.linear_fwd(x3, dev["w"], dev["b"], dev["res"][None], act=ms.ACT_GELU)
    assert got.shape == (1, M, 96) and torch().equal(got[0], want)


@pytest.mark.parametrize("M", [4, 500])
def test_nan_and_infinity_stay_in_their_rows(M):
    dev, ref = make(M, 72, 80, "bf16", 12)
    dev["x"][1, 71] = float("nan")
    dev["x"][M - 1, 0] = float("inf")
    out, _ = ms.linear_fwd(dev["x"], dev["w"], dev["b"], dev["res"], act=ms.ACT_SILU)
    want, _ = linear_ref(ref["x"], ref["w"], ref["b"], ref["res"], "silu")
    got = from_dev(out)
    assert np.all(np.isnan(got[1]))
    good = [m for m in range(M) if m not in (1, M - 1)]
    close("rows", got[good], want[good], "bf16")


def test_gradients_against_differences():
    """Central differences of the kernel's forward along the gradient's signs; float32 rounding over the step leaves
    about 1e-3 of the derivative, 1e-2 is asked.  Not for relu: a step moves a row's products by up to 0.1 here, over
    the kink of one in twenty of them, and a difference over a kink is no derivative; relu's gradient is held to the
    formula above and, in float64, to differences with a step that crosses none."""
    for act in ("none", "silu", "gelu"):
        for M in (20, 150):
            dev, _ = make(M, 72, 56, "f32", 13)

            def loss(v):
                out, _ = ms.linear_fwd(v["x"], v["w"], v["b"], act=ACTS[act])
                return float((out.double() * v["dout"].double()).sum())

            _, pre = ms.linear_fwd(dev["x"], dev["w"], dev["b"], act=ACTS[act], want_pre=True)
            g = ms.linear_bwd(dev["x"], dev["w"], dout=dev["dout"], pre=pre, act=ACTS[act])
            for k, gk in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
                d = torch().sign(g[gk])
                eps = 2e-3
                up, down = dict(dev), dict(dev)
                up[k], down[k] = dev[k] + eps * d, dev[k] - eps * d
                num = (loss(up) - loss(down)) / (2 * eps)
                want = float((g[gk].double() * d.double()).sum())
                assert abs(num - want) <= 1e-2 * abs(want), (act, M, k, num, want)


def test_other_stream_and_graph():
    t = torch()
    for M in (6, 300):
        dev, _ = make(M, 1032, 264, "bf16", 14)
        a = (dev["x"], dev["w"], dev["b"], dev["res"])
        want = ms.linear_fwd(*a, act=ms.ACT_SILU, want_pre=True)
        wg = ms.linear_bwd(*a[:2], dout=dev["dout"], pre=want[1], act=ms.ACT_SILU)
        t.cuda.synchronize()
        s = t.cuda.Stream()
        got = ms.linear_fwd(*a, act=ms.ACT_SILU, want_pre=True, stream=s)
        g = ms.linear_bwd(*a[:2], dout=dev["dout"], pre=got[1], act=ms.ACT_SILU, stream=s)
        s.synchronize()
        assert all(t.equal(x, y) for x, y in zip(got, want)) and all(t.equal(g[k], wg[k]) for k in g)
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            got = ms.linear_fwd(*a, act=ms.ACT_SILU, want_pre=True)
            g = ms.linear_bwd(*a[:2], dout=dev["dout"], pre=got[1], act=ms.ACT_SILU)
        for _ in range(3):
            for v in list(got) + list(g.values()):
                v.zero_()
            graph.replay()
            t.cuda.synchronize()
            assert all(t.equal(x, y) for x, y in zip(got, want)) and all(t.equal(g[k], wg[k]) for k in g)
            junk = t.randn(1 << 20, device="cuda:0").sum().item()
            assert junk == junk


def test_binding_refusals():
    t = torch()
    x, w = t.zeros(4, 64, device="cuda:0"), t.zeros(32, 64, device="cuda:0")
    with pytest.raises(ValueError):
        ms.linear_fwd(x, w[:, :56].contiguous())
    with pytest.raises(ValueError):
        ms.linear_fwd(x, t.zeros(64, 32, device="cuda:0").t())
    with pytest.raises(TypeError):
        ms.linear_fwd(x, w.bfloat16())
    with pytest.raises(TypeError):
        ms.linear_fwd(x.half(), w.half())
    with pytest.raises(ValueError):
        ms.linear_fwd(x, w, residual=t.zeros(4, 31, device="cuda:0"))
    with pytest.raises(ms.MambaError):
        ms.linear_fwd(x[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(ms.MambaError):
        ms.linear_fwd(x, w, act=7)
    with pytest.raises(ms.MambaError):  # the activation's derivative needs pre
        ms.linear_bwd(x, w, dout=t.zeros(4, 32, device="cuda:0"), act=ms.ACT_SILU)
    with pytest.raises(ms.MambaError):
        ms.linear_fwd(x[:0], w)

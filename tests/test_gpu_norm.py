"""GPU parity of group normalisation with an activation (mamba_group_norm_*,
through the C ABI) with its plain float64 form: groups that begin and end inside
a vector of 8 channels, one group, a group a channel, single tokens, maps of
several runs of rows with a short last one, many items, and each activation.

Tolerances, written before the first run.  Sums of n values about a value of
their own, in float32, err by a few sqrt(n)·2^-24 of their scale, so statistics
and float32 outputs are held to the project's 2e-4 (normwise) and 2e-5 (L2);
bfloat16 outputs to 1e-2 and 3e-3.  Sums over all items (dweight, dbias) cancel
to about sqrt(N) of N terms: 2e-4 of their largest value covers N up to 1e6.

With all values of a group equal, dx is rstd times a difference that vanishes."""
import numpy as np
import pytest

import selective_state_space_mamba_amd as ms

from layerutil import ACTS, from_dev, norm_ref, rounded, to_dev
from scanutil import errors, torch

pytestmark = pytest.mark.gpu
TOL = {"f32": (2e-4, 2e-5), "bf16": (1e-2, 3e-3), "sum": (2e-4, 2e-4)}


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


def make(B, L, D, dtype, seed, offset=1.0):
    r = np.random.Generator(np.random.PCG64([seed, 5]))
    v = {}
    v["x"] = rounded(r.standard_normal((B, L, D)) + offset * r.standard_normal(D), dtype)
    v["dout"] = rounded(r.standard_normal((B, L, D)), dtype)
    for k, m in (("w", 1.0), ("b", 0.0)):
        a = (m + 0.2 * r.standard_normal(D)).astype(np.float32)
        v[k] = (a, a.astype(np.float64))
    return {k: to_dev(a) for k, (a, _) in v.items()}, {k: f for k, (_, f) in v.items()}


CASES = [
    # B, L, D, G, dtype, act
    (1, 1, 8, 1, "f32", "none"),
    (3, 1, 1536, 24, "bf16", "none"),
    (3, 1, 1536, 1, "f32", "silu"),
    (5, 1, 192, 32, "bf16", "gelu"),
    (2, 1, 2048, 1, "bf16", "relu"),
    (4, 7, 64, 64, "f32", "silu"),
    (2, 49, 72, 24, "bf16", "silu"),
    (2, 49, 8192, 8, "f32", "gelu"),
    (2, 33, 5000, 1, "bf16", "silu"),
    (3, 1001, 192, 32, "bf16", "silu"),
    (1, 4099, 96, 4, "f32", "gelu"),
    (2, 2500, 40, 1, "f32", "relu"),
    (1, 300, 2056, 257, "f32", "none"),
    (2500, 3, 24, 3, "bf16", "silu"),
    (3000, 1, 64, 8, "f32", "gelu"),
    (1030, 40, 16, 2, "f32", "silu"),
    # single tokens: each vector width, several vectors a lane, groups too wide for a lane group
    (7, 1, 40, 8, "bf16", "silu"),
    (5000, 1, 48, 12, "f32", "relu"),
    (70, 1, 1032, 3, "f32", "silu"),
    (9, 1, 4128, 3, "bf16", "gelu"),
    (4, 1, 8192, 1, "f32", "silu"),
    (4, 1, 8192, 2, "bf16", "none"),
    (3, 1, 3000, 8, "f32", "silu"),
    (3, 1, 1000, 8, "bf16", "silu"),
    (9000, 1, 256, 4, "bf16", "none"),
    # single tokens through LDS: odd groups and pairs and fours, short last workgroups, lane groups that
    # begin anywhere among a token's groups and take many rows, one workgroup's lane group a wave
    (3001, 1, 24, 8, "bf16", "relu"),
    (2000, 1, 408, 8, "bf16", "gelu"),
    (601, 1, 2040, 8, "f32", "silu"),
    (999, 1, 240, 40, "bf16", "silu"),
    (33, 1, 4008, 4, "bf16", "none"),
    (33, 1, 1800, 2, "f32", "gelu"),
    (20000, 1, 1224, 24, "bf16", "silu"),
    (1, 1, 1096, 8, "f32", "none"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B%d-L%d-D%d-G%d-%s-%s" % c)
def test_forward_and_gradients(case):
    B, L, D, G, dtype, act = case
    print("[gpu case] norm", case, flush=True)
    dev, ref = make(B, L, D, dtype, L + D)
    out, mean, rstd = ms.group_norm_fwd(dev["x"], G, dev["w"], dev["b"], eps=1e-5, act=ACTS[act])
    g = ms.group_norm_bwd(dev["x"], G, dev["w"], dev["b"], dout=dev["dout"], mean=mean, rstd=rstd, act=ACTS[act])
    torch().cuda.synchronize()
    want, wm, wr, wg = norm_ref(ref["x"], G, ref["w"], ref["b"], act, 1e-5, ref["dout"])
    close("mean", from_dev(mean), wm, "f32")
    if L * D // G > 1:
        close("rstd", from_dev(rstd), wr, "f32")
    close("out", from_dev(out), want, dtype)
    close("dx", from_dev(g["dx"]), wg["dx"], dtype)
    close("dweight", from_dev(g["dweight"]), wg["dweight"], "sum")
    close("dbias", from_dev(g["dbias"]), wg["dbias"], "sum")
    again = ms.group_norm_bwd(dev["x"], G, dev["w"], dev["b"], dout=dev["dout"], mean=mean, rstd=rstd, act=ACTS[act])
    assert all(torch().equal(g[k], again[k]) for k in g)


def test_without_weight_and_bias():
    for B, L, D, G in ((2, 1, 64, 8), (2, 900, 64, 8)):
        dev, ref = make(B, L, D, "f32", 3)
        out, mean, rstd = ms.group_norm_fwd(dev["x"], G, act=ms.ACT_SILU)
        g = ms.group_norm_bwd(dev["x"], G, dout=dev["dout"], mean=mean, rstd=rstd, act=ms.ACT_SILU)
        want, _, _, wg = norm_ref(ref["x"], G, None, None, "silu", 1e-5, ref["dout"])
        close("out", from_dev(out), want, "f32")
        close("dx", from_dev(g["dx"]), wg["dx"], "f32")
        assert g["dweight"] is None and g["dbias"] is None


@pytest.mark.parametrize("L", [1, 9, 3000])
def test_large_offsets_and_constant_groups(L):
    """Channels 1000 standard deviations from zero (in float32 a value keeps 6e-5 of its deviation, an output so much
    of its scale), and a group without any variance, whose output is the bias and whose gradient stays finite."""
    B, D, G = 2, 64, 4
    r = np.random.Generator(np.random.PCG64(8))
    x = (r.standard_normal((B, L, D)) + 1000.0).astype(np.float32)
    x[:, :, :16] = 7.25
    w, b = r.standard_normal(D).astype(np.float32), r.standard_normal(D).astype(np.float32)
    dout = r.standard_normal((B, L, D)).astype(np.float32)
    out, mean, rstd = ms.group_norm_fwd(to_dev(x), G, to_dev(w), to_dev(b))
    g = ms.group_norm_bwd(to_dev(x), G, to_dev(w), to_dev(b), dout=to_dev(dout), mean=mean, rstd=rstd)
    want, _, _ = norm_ref(x.astype(np.float64), G, w.astype(np.float64), b.astype(np.float64), "none", 1e-5)
    assert np.max(np.abs(from_dev(out) - want)) <= 1e-3 * np.max(np.abs(want))
    assert np.array_equal(from_dev(out)[:, :, :16], np.broadcast_to(b[:16].astype(np.float64), (B, L, 16)))
    assert all(np.all(np.isfinite(from_dev(v))) for v in g.values())


@pytest.mark.parametrize("L", [1, 2000])
def test_nan_and_infinity_stay_in_their_group(L):
    dev, ref = make(2, L, 48, "f32", 4)
    dev["x"][0, L // 2, 13] = float("nan")  # group 2 of 8: channels 12..17
    dev["x"][1, L - 1, 0] = float("inf")    # group 0
    out, mean, rstd = ms.group_norm_fwd(dev["x"], 8, dev["w"], dev["b"], act=ms.ACT_SILU)
    want, _, _ = norm_ref(ref["x"], 8, ref["w"], ref["b"], "silu", 1e-5)
    got = from_dev(out).reshape(2, L, 8, 6)
    want = want.reshape(2, L, 8, 6)
    bad = {(0, 2), (1, 0)}
    for b in range(2):
        for k in range(8):
            if (b, k) in bad:
                assert np.all(np.isnan(got[b, :, k]))
            else:
                close("group", got[b, :, k], want[b, :, k], "f32")


def test_gradients_against_differences():
    """Central differences of the kernel's forward along the gradient's signs; float32 rounding over the step leaves
    about 1e-3 of the derivative, 1e-2 is asked."""
    for act in ACTS:
        dev, _ = make(2, 60, 48, "f32", 6)

        def loss(v):
            out, _, _ = ms.group_norm_fwd(v["x"], 8, v["w"], v["b"], act=ACTS[act])
            return float((out.double() * v["dout"].double()).sum())

        _, mean, rstd = ms.group_norm_fwd(dev["x"], 8, dev["w"], dev["b"], act=ACTS[act])
        g = ms.group_norm_bwd(dev["x"], 8, dev["w"], dev["b"], dout=dev["dout"], mean=mean, rstd=rstd, act=ACTS[act])
        for k, gk in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
            d = torch().sign(g[gk])
            eps = 2e-3
            up, down = dict(dev), dict(dev)
            up[k], down[k] = dev[k] + eps * d, dev[k] - eps * d
            num = (loss(up) - loss(down)) / (2 * eps)
            want = float((g[gk].double() * d.double()).sum())
            assert abs(num - want) <= 1e-2 * abs(want), (act, k, num, want)


def test_other_stream_and_graph():
    t = torch()
    for L in (1, 3000):
        dev, _ = make(4, L, 192, "bf16", 7)
        a = (dev["x"], 32, dev["w"], dev["b"])
        want = ms.group_norm_fwd(*a, act=ms.ACT_SILU)
        wg = ms.group_norm_bwd(*a, dout=dev["dout"], mean=want[1], rstd=want[2], act=ms.ACT_SILU)
        t.cuda.synchronize()
        s = t.cuda.Stream()
        got = ms.group_norm_fwd(*a, act=ms.ACT_SILU, stream=s)
        g = ms.group_norm_bwd(*a, dout=dev["dout"], mean=got[1], rstd=got[2], act=ms.ACT_SILU, stream=s)
        s.synchronize()
        assert all(t.equal(x, y) for x, y in zip(got, want)) and all(t.equal(g[k], wg[k]) for k in g)
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            got = ms.group_norm_fwd(*a, act=ms.ACT_SILU)
            g = ms.group_norm_bwd(*a, dout=dev["dout"], mean=got[1], rstd=got[2], act=ms.ACT_SILU)
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
    x = t.zeros(2, 8, 64, device="cuda:0")
    with pytest.raises(ms.MambaError):
        ms.group_norm_fwd(x, 5)
    with pytest.raises(ms.MambaError):
        ms.group_norm_fwd(x, 4, act=9)
    with pytest.raises(ms.MambaError):
        ms.group_norm_fwd(x[:, :, :12].contiguous(), 3)
    with pytest.raises(ValueError):
        ms.group_norm_fwd(x, 4, t.ones(63, device="cuda:0"))
    with pytest.raises(TypeError):
        ms.group_norm_fwd(x, 4, t.ones(64, device="cuda:0", dtype=t.bfloat16))
    with pytest.raises(ValueError):
        ms.group_norm_fwd(x[:, :, ::2], 4)
    with pytest.raises(TypeError):
        ms.group_norm_fwd(x.half(), 4)

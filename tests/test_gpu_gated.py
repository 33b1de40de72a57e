"""GPU parity of the gated pair of products (mamba_gated_linear_*) with its
float64 form: one row, both sides of the few-rows kernel's limits, sizes that
end inside every tile and stage, split contractions, each activation, each
gradient alone.  Tolerances: ffutil's, derived there."""
import pytest

import selective_state_space_mamba_amd as ms

from ffutil import close, gated_ref, maker, planned_kind
from layerutil import ACTS
from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


def make(M, K, N, dtype, seed, bias=(True, True)):
    n = maker(seed)
    return dict(x=n((M, K), dtype), wg=n((N, K), dtype, K ** -0.5), wu=n((N, K), dtype, K ** -0.5),
                bg=n((N,), std=0.2) if bias[0] else None, bu=n((N,), std=0.2) if bias[1] else None,
                dout=n((M, N), dtype))


CASES = [
    # M, K, N, dtype, act, biases
    (1, 8, 8, "f32", "none", (True, True)),
    (1, 8, 8, "bf16", "silu", (False, True)),
    (1, 1536, 768, "bf16", "silu", (False, False)),
    (8, 1000, 24, "f32", "gelu", (True, False)),
    (15, 72, 200, "bf16", "relu", (True, True)),
    (17, 4096, 40, "bf16", "silu", (False, False)),
    (32, 264, 1032, "bf16", "silu", (True, True)),     # bias sums of one run of rows
    (31, 40, 520, "f32", "gelu", (True, True)),
    (33, 264, 1032, "f32", "silu", (True, True)),
    (64, 40, 136, "bf16", "gelu", (True, True)),
    (65, 40, 136, "bf16", "gelu", (True, True)),
    (127, 8, 8, "bf16", "none", (False, False)),
    (129, 72, 136, "f32", "relu", (True, True)),
    (128, 128, 64, "bf16", "none", (False, False)),
    (200, 2056, 264, "bf16", "silu", (True, False)),   # blocks of few rows; in dx and dw, shares of the contraction
    (300, 4104, 264, "bf16", "silu", (True, True)),    # shares of the contraction in the forward too
    (250, 520, 4104, "bf16", "relu", (False, True)),
    (200, 2056, 264, "f32", "gelu", (False, True)),
    (1000, 200, 96, "f32", "none", (True, True)),
    (70, 136, 48, "f32", "silu", (True, True)),
    (90, 72, 32, "bf16", "silu", (True, True)),
    (1500, 768, 1544, "bf16", "silu", (True, True)),
    (5003, 520, 256, "bf16", "gelu", (True, True)),
    (2100, 264, 1048, "bf16", "relu", (False, False)),
    (16300, 328, 776, "bf16", "silu", (True, True)),   # enough tiles for the large ones, the last partly empty
    (4100, 1000, 2056, "bf16", "silu", (False, False)),
    (3000, 96, 56, "f32", "silu", (True, True)),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%dx%d-%s-%s-b%s" % c)
def test_forward_and_gradients(case):
    M, K, N, dtype, act, bias = case
    print("[gpu case] gated", case, flush=True)
    t = torch()
    v = make(M, K, N, dtype, M + K + N, bias)
    out, pre = ms.gated_linear_fwd(v["x"], v["wg"], v["wu"], v["bg"], v["bu"], act=ACTS[act], want_pre=True)
    bare, none = ms.gated_linear_fwd(v["x"], v["wg"], v["wu"], v["bg"], v["bu"], act=ACTS[act])
    assert none is None and t.equal(bare, out)
    g = ms.gated_linear_bwd(v["x"], v["wg"], v["wu"], dout=v["dout"], pre=pre, act=ACTS[act])
    want, wg, wu, grads = gated_ref(v["x"], v["wg"], v["wu"], v["bg"], v["bu"], act, v["dout"])
    close("out", out, want, dtype)
    close("gate", pre[0], wg, "f32")
    close("up", pre[1], wu, "f32")
    for k in grads:
        close(k, g[k], grads[k], "f32" if dtype == "f32" or k[:2] == "db" else "bf16 grad")
    again = ms.gated_linear_bwd(v["x"], v["wg"], v["wu"], dout=v["dout"], pre=pre, act=ACTS[act])
    assert all(t.equal(g[k], again[k]) for k in g)
    for want_k, keys in (("want_dx", ("dx",)), ("want_dweight", ("dw_gate", "dw_up")), ("want_dbias", ("db_gate", "db_up"))):
        kw = dict(want_dx=False, want_dweight=False, want_dbias=False)
        kw[want_k] = True
        one = ms.gated_linear_bwd(v["x"], v["wg"], v["wu"], dout=v["dout"], pre=pre, act=ACTS[act], **kw)
        assert all(t.equal(one[k], g[k]) if k in keys else one[k] is None for k in g)


def test_exact_products():
    """Small whole numbers: every sum is exact in float32, so the tiles' layout shows without a tolerance."""
    t = torch()
    gen = t.Generator(device="cpu")
    gen.manual_seed(1)

    def ints(lo, hi, *shape):
        return t.randint(lo, hi, shape, generator=gen).double().to("cuda:0")

    for dtype in (t.float32, t.bfloat16):
        for M, K, N in ((5, 48, 32), (130, 88, 72), (300, 1032, 136), (600, 136, 264), (16400, 72, 1032)):
            x, wg, wu = ints(-2, 3, M, K), ints(-1, 2, N, K), ints(-1, 2, N, K)
            wg[:, 8:] = 0  # gates of at most 16, whole
            dout = ints(-1, 2, M, N)
            a = [v.to(dtype) for v in (x, wg, wu, dout)]
            out, pre = ms.gated_linear_fwd(a[0], a[1], a[2], act=ms.ACT_RELU, want_pre=True)
            want, g, u = gated_ref(x, wg, wu, None, None, "relu")
            assert t.equal(pre[0].double(), g) and t.equal(pre[1].double(), u)
            assert t.equal(out, want.float().to(dtype))
            if dtype is t.bfloat16:  # what enters the products is exact up to 256
                keep = (u.abs() <= 256) & (g.abs() <= 256)
                a[3] = (dout * keep).to(dtype)
            got = ms.gated_linear_bwd(*a[:3], dout=a[3], pre=pre, act=ms.ACT_RELU)
            grads = gated_ref(x, wg, wu, None, None, "relu", a[3].double())[3]
            for k, v in grads.items():
                assert float(v.abs().max()) < 1 << 24
                assert t.equal(got[k], v.float().to(got[k].dtype)), (dtype, M, K, N, k)


# Sizes at which the three products of the pair take each tile, whole and in shares of the contraction.
TILED = [(300, 136, 64), (300, 136, 512), (1000, 136, 64), (300, 1024, 4104), (300, 1536, 4104), (700, 4104, 4104),
         (8192, 136, 4104), (16384, 136, 2048), (16384, 200, 4104), (40000, 136, 64), (40000, 136, 128), (9000, 136, 1032),
         (300, 1040, 64), (300, 1040, 72), (400, 4112, 4104), (100, 4112, 64), (300, 528, 64), (300, 528, 200),
         (130, 8208, 4104)]


def test_every_tile():
    """Whole numbers through every tile of the forward (128 and 256 columns, and the long one), of dx (as the plain product with twice the rows of a weight, whole stages each)
    and dW (with 2N rows), without a tolerance; and that TILED is what the comment says."""
    t = torch()
    gen = t.Generator(device="cpu")
    gen.manual_seed(4)
    seen = set()
    for M, K, N in TILED:
        print("[gpu case] gated tiles", M, K, N, flush=True)
        stages = -(-N // 64) * 64
        for product, dims in ((1, ms.make_linear_dims(M, K, 2 * stages, ms.DTYPE_BF16)),
                              (2, ms.make_linear_dims(M, K, 2 * N, ms.DTYPE_BF16))):
            rows, cols, shares = ms.linear_plan(dims, product)
            seen.add((product, rows, cols, shares > 1))
        kind = planned_kind("gated", M, K, N)
        seen.add((0,) + (kind if kind[0] == "long" else kind[1:3] + (kind[3] > 1,)))

        def ints(lo, hi, *shape):
            return t.randint(lo, hi, shape, generator=gen).double().to("cuda:0")

        x, wg, wu = ints(-2, 3, M, K), ints(-1, 2, N, K), ints(-1, 2, N, K)
        wg[:, 8:] = 0
        wu[:, 60:] = 0  # factors that bfloat16 holds
        dout = ints(-1, 2, M, N)
        a = [v.bfloat16() for v in (x, wg, wu, dout)]
        out, pre = ms.gated_linear_fwd(a[0], a[1], a[2], act=ms.ACT_RELU, want_pre=True)
        want, g, u, grads = gated_ref(x, wg, wu, None, None, "relu", dout)
        assert t.equal(pre[0].double(), g) and t.equal(pre[1].double(), u) and t.equal(out, want.float().bfloat16())
        assert float(u.abs().max()) <= 256
        got = ms.gated_linear_bwd(a[0], a[1], a[2], dout=a[3], pre=pre, act=ms.ACT_RELU)
        for k, v in grads.items():
            assert float(v.abs().max()) < 1 << 24
            assert t.equal(got[k], v.float().to(got[k].dtype)), (M, K, N, k)
    tiles = [(128, 128), (256, 192), (256, 256)]
    assert seen >= {(p,) + tile + (split,) for p in (0, 1, 2) for tile in tiles for split in (False, True)
                    if p > 0 or tile != (256, 192)} | {(0, "long", 4), (0, "long", 8)}, seen


@pytest.mark.parametrize("M,K", [(4, 72), (500, 72), (500, 1096)])
def test_rows_stay_apart_and_stacked_weights(M, K):
    t = torch()
    v = make(M, K, 80, "bf16", 12)
    v["x"][1, 71] = float("nan")
    v["x"][M - 1, 0] = float("inf")
    args = (v["wg"], v["wu"], v["bg"], v["bu"])
    out, _ = ms.gated_linear_fwd(v["x"], *args)
    assert bool(out[1].isnan().all())
    good = [m for m in range(M) if m not in (1, M - 1)]
    want, _, _ = gated_ref(v["x"][good], *args, "silu")
    close("rows", out[good], want, "bf16")
    both = t.cat([v["wg"], v["wu"]])  # halves of one weight
    got, _ = ms.gated_linear_fwd(v["x"][None], both[:80], both[80:], v["bg"], v["bu"])
    assert got.shape == (1, M, 80) and t.equal(got[0].view(t.int16), out.view(t.int16))


def test_gradients_against_differences():
    """Central differences of the kernel's float32 forward along the gradient's signs: rounding over the step leaves
    about 1e-3 of the derivative, 1e-2 is asked.  (Not for relu, whose kink a step would cross.)"""
    t = torch()
    for act in ("none", "silu", "gelu"):
        for M in (20, 150):
            v = make(M, 72, 56, "f32", 13)

            def loss(s):
                out, _ = ms.gated_linear_fwd(s["x"], s["wg"], s["wu"], s["bg"], s["bu"], act=ACTS[act])
                return float((out.double() * s["dout"].double()).sum())

            _, pre = ms.gated_linear_fwd(v["x"], v["wg"], v["wu"], v["bg"], v["bu"], act=ACTS[act], want_pre=True)
            g = ms.gated_linear_bwd(v["x"], v["wg"], v["wu"], dout=v["dout"], pre=pre, act=ACTS[act])
            for k, gk in (("x", "dx"), ("wg", "dw_gate"), ("wu", "dw_up"), ("bg", "db_gate"), ("bu", "db_up")):
                d = t.sign(g[gk])
                eps = 1e-3
                num = (loss(dict(v, **{k: v[k] + eps * d})) - loss(dict(v, **{k: v[k] - eps * d}))) / (2 * eps)
                want = float((g[gk].double() * d.double()).sum())
                assert abs(num - want) <= 1e-2 * abs(want), (act, M, k, num, want)


def test_other_stream_and_graph():
    t = torch()
    for M in (6, 300):
        v = make(M, 1032, 264, "bf16", 14)

        def both(**kw):
            out, pre = ms.gated_linear_fwd(v["x"], v["wg"], v["wu"], v["bg"], v["bu"], want_pre=True, **kw)
            g = ms.gated_linear_bwd(v["x"], v["wg"], v["wu"], dout=v["dout"], pre=pre, **kw)
            return [out, pre] + list(g.values())

        want = both()
        t.cuda.synchronize()
        s = t.cuda.Stream()
        got = both(stream=s)
        s.synchronize()
        assert all(t.equal(a, b) for a, b in zip(got, want))
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            got = both()
        n = maker(M)
        for k in range(3):
            for b in got:
                b.zero_()
            v["x"].copy_(n((M, 1032), "bf16"))
            graph.replay()
            t.cuda.synchronize()
            junk = t.randn(1 << 20, device="cuda:0").sum().item()
            assert junk == junk
            assert all(t.equal(a, b) for a, b in zip(got, both())), k


def test_more_elements_than_32_bits_count():
    """pre of more than 2^32 values: the last rows against a call of their own."""
    t = torch()
    M, K, N = 270000, 16, 8192
    print("[gpu case] gated sizes", M, K, N, flush=True)
    v = make(256, K, N, "bf16", 3, (False, False))
    x = v["x"].repeat(M // 256 + 1, 1)[:M].contiguous()
    out, pre = ms.gated_linear_fwd(x, v["wg"], v["wu"], want_pre=True)
    want, wpre = ms.gated_linear_fwd(v["x"], v["wg"], v["wu"], want_pre=True)
    tail = M % 256
    assert t.equal(out[-tail:], want[:tail]) and t.equal(pre[:, -tail:], wpre[:, :tail]) and t.equal(out[:256], want)
    dout = v["dout"].repeat(M // 256 + 1, 1)[:M].contiguous()
    g = ms.gated_linear_bwd(x, v["wg"], v["wu"], dout=dout, pre=pre, want_dweight=False, want_dbias=False)
    wx = gated_ref(v["x"], v["wg"], v["wu"], None, None, "silu", v["dout"])[3]["dx"]
    close("dx", g["dx"][-tail:], wx[:tail], "bf16 grad")
    close("dx", g["dx"][:256], wx, "bf16 grad")


def test_binding_refusals():
    t = torch()
    z = lambda *s, dtype=t.float32: t.zeros(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    x, w = z(4, 64), z(32, 64)
    for bad in ((x, w, z(40, 64)), (x, w[:, :56].contiguous(), w), (x, z(64, 32).t(), w)):
        with pytest.raises(ValueError):
            ms.gated_linear_fwd(*bad)
    with pytest.raises(TypeError):
        ms.gated_linear_fwd(x, w, w.bfloat16())
    with pytest.raises(ValueError):
        ms.gated_linear_fwd(x, w, w, z(31))
    with pytest.raises(TypeError):
        ms.gated_linear_fwd(x, w, w, None, z(32, dtype=t.bfloat16))
    with pytest.raises(ms.MambaError):
        ms.gated_linear_fwd(x, w, w, act=5)
    with pytest.raises(ms.MambaError):
        ms.gated_linear_fwd(x[:0], w, w)
    with pytest.raises(ms.MambaError):
        ms.gated_linear_fwd(x[:, :60].contiguous(), w[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(ValueError):
        ms.gated_linear_bwd(x, w, w, dout=z(4, 32), pre=z(4, 32))
    with pytest.raises(ms.MambaError):
        ms.gated_linear_bwd(x, w, w, dout=z(4, 32), pre=z(2, 4, 32), want_dx=False, want_dweight=False, want_dbias=False)

"""GPU parity of the products with quantised weights (mamba_linear_q8,
mamba_linear_q4) with their float64 forms: one row, both sides of the few-rows
kernels' limits, sizes that end inside every tile, turn and group, each
activation.  Tolerances: ffutil's, derived there (products of 8- and 4-bit
values are exact in float32; the sums of 1 + q/128 before the zero is taken off
are some 30 times the result: 30·sqrt(128)·2^-24 = 2e-5 of a group's, less by
the root of the groups' number, in L2 below 1e-5)."""
import pytest

import selective_state_space_mamba_amd as ms

from ffutil import close, dtype_of, finish_ref, maker, mm, planned_kind, rows8, weights4
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


def want8(q, sx, w, sw, b, act, res):
    return finish_ref(mm(q.float(), w.float()) * sx.double()[:, None] * sw.double(), b, act, res)


Q8 = [
    # M, K, N, dtype, act, bias, residual
    (1, 16, 8, "f32", "none", False, False), (1, 16, 8, "bf16", "silu", True, True), (1, 4096, 768, "bf16", "none", True, True),
    (8, 1008, 24, "f32", "gelu", False, True), (15, 80, 200, "bf16", "relu", True, True), (17, 4096, 40, "bf16", "silu", True, False),
    (33, 272, 1032, "f32", "silu", True, True), (64, 48, 136, "bf16", "gelu", True, True), (65, 48, 136, "bf16", "gelu", True, True),
    (127, 16, 8, "bf16", "none", False, False), (129, 144, 136, "f32", "relu", True, True), (128, 128, 128, "bf16", "none", False, False),
    (200, 4112, 264, "bf16", "silu", True, True), (200, 4112, 264, "f32", "gelu", True, True), (1000, 208, 96, "f32", "none", True, False),
    (300, 8208, 264, "bf16", "silu", True, True), (300, 8208, 264, "f32", "gelu", True, True), (250, 1040, 4104, "bf16", "none", True, True),
    (1500, 768, 1544, "bf16", "silu", True, False), (5003, 528, 256, "bf16", "gelu", True, True),
    (16300, 656, 1528, "bf16", "silu", True, True), (16300, 656, 1528, "f32", "silu", True, True),
    (8200, 2000, 2056, "bf16", "none", True, True), (8200, 2000, 2056, "f32", "none", True, True),
]


@pytest.mark.parametrize("case", Q8, ids=lambda c: "%dx%dx%d-%s-%s-b%d-r%d" % c)
def test_8bit(case):
    M, K, N, dtype, act, bias, res = case
    print("[gpu case] q8", case, flush=True)
    n = maker(M + K + N)
    x, sx = rows8(n((M, K)))
    w, sw = rows8(n((N, K)))
    sw = sw * K ** -0.5
    b, r = n((N,), std=0.2) if bias else None, n((M, N), dtype) if res else None
    got = ms.linear_q8(x, sx, w, sw, b, r, act=ACTS[act], dtype=dtype_of(dtype))
    assert got.dtype is dtype_of(dtype)
    close("out", got, want8(x, sx, w, sw, b, act, r), dtype)
    again = ms.linear_q8(x, sx, w, sw, b, r, act=ACTS[act], dtype=dtype_of(dtype))
    assert torch().equal(got, again)
    if res:
        buf = r.clone()
        assert ms.linear_q8(x, sx, w, sw, b, buf, act=ACTS[act], out=buf) is buf and torch().equal(buf, got)


def test_8bit_exact_products():
    """Whole numbers and every e4m3 value: sums exact in float32, so layout and formats show without a tolerance."""
    t = torch()
    gen = t.Generator(device="cpu")
    gen.manual_seed(2)
    for M, K, N in ((5, 48, 32), (40, 304, 40), (130, 144, 72), (300, 2064, 136), (2100, 272, 1032), (16400, 144, 1032)):
        x = t.randint(-3, 4, (M, K), generator=gen).float().to("cuda:0")
        w = t.randint(-2, 3, (N, K), generator=gen).float().to("cuda:0")
        sx = 2.0 ** t.randint(-3, 4, (M,), generator=gen).float().to("cuda:0")
        sw = 2.0 ** t.randint(-3, 4, (N,), generator=gen).float().to("cuda:0")
        got = ms.linear_q8(x.to(t.float8_e4m3fn), sx, w.to(t.float8_e4m3fn), sw, dtype=t.float32)
        assert t.equal(got.double(), mm(x, w) * sx.double()[:, None] * sw.double()), (M, K, N)
    # every finite value in every place of a stage, against one column of ones a row
    codes = t.arange(256, dtype=t.uint8, device="cuda:0")
    codes = codes[(codes & 127) != 127]
    for M in (254, 5):  # tiles; few rows
        x = codes[t.arange(M * 256, device="cuda:0").view(M, 256) * 37 % 254].view(t.float8_e4m3fn)
        w = t.eye(256, device="cuda:0").to(t.float8_e4m3fn)
        one = t.ones(256, device="cuda:0")
        got = ms.linear_q8(x, one[:1].expand(M).contiguous(), w, one, dtype=t.float32)
        assert t.equal(got, x.float())


# Sizes at which the product takes each tile, whole and in shares of the contraction, and the long one.
TILED = [(300, 144, 64), (300, 2064, 64), (40000, 528, 136), (1000, 8208, 4104), (40000, 144, 136), (400, 8208, 8200),
         (2000, 144, 6152), (9000, 12304, 136), (100, 12304, 64), (300, 528, 64), (300, 528, 72), (1000, 4112, 200)]


def test_8bit_every_tile():
    """Whole numbers through every tile, without a tolerance, for both types of output; and that TILED is what the
    comment says."""
    t = torch()
    gen = t.Generator(device="cpu")
    gen.manual_seed(3)
    seen = set()
    for M, K, N in TILED:
        print("[gpu case] q8 tiles", M, K, N, flush=True)
        kind = planned_kind("q8", M, K, N)
        seen.add(kind if kind[0] == "long" else kind[1:3] + (kind[3] > 1,))
        x = t.randint(-1, 2, (M, K), generator=gen).float().to("cuda:0")
        w = t.randint(-1, 2, (N, K), generator=gen).float().to("cuda:0")
        res = t.randint(-9, 10, (M, N), generator=gen).float().to("cuda:0")
        sx, sw = t.full((M,), 0.5, device="cuda:0"), t.full((N,), 2.0, device="cuda:0")
        want = mm(x, w) + res.double()
        for dt in (t.float32, t.bfloat16):
            got = ms.linear_q8(x.to(t.float8_e4m3fn), sx, w.to(t.float8_e4m3fn), sw, None, res.to(dt))
            assert t.equal(got, want.float().to(dt)), (M, K, N, dt)
    assert seen == {tile + (split,) for tile in ((128, 128), (256, 192), (256, 256)) for split in (False, True)} | {
        ("long", 4), ("long", 8)}, seen


@pytest.mark.parametrize("M,K", [(4, 96), (300, 96), (300, 528)])
def test_8bit_rows_stay_apart(M, K):
    t = torch()
    n = maker(M)
    x, sx = rows8(n((M, K)))
    w, sw = rows8(n((40, K)))
    x.view(t.uint8)[1, 5] = 0x7f  # NaN
    sx[M - 1] = 0
    got = ms.linear_q8(x, sx, w, sw)
    assert bool(got[1].isnan().all()) and bool((got[M - 1] == 0).all())
    good = [m for m in range(M) if m != 1]
    close("rows", got[good], want8(x, sx, w, sw, None, "none", None)[good], "bf16")


Q4 = [
    # M, K, N, dtype, scale's type, group, zero, act, bias, residual
    (1, 32, 8, "bf16", "bf16", 32, False, "none", False, False), (1, 32, 8, "f32", "f32", 128, True, "none", True, True),
    (1, 4096, 768, "bf16", "bf16", 128, False, "none", False, True), (1, 4096, 768, "bf16", "f32", 128, True, "silu", True, False),
    (2, 96, 24, "bf16", "bf16", 64, True, "relu", True, True), (7, 1056, 200, "f32", "f32", 32, True, "gelu", True, True),
    (16, 2080, 264, "bf16", "bf16", 32, True, "silu", True, True), (17, 2080, 264, "bf16", "bf16", 64, False, "none", True, False),
    (32, 160, 1032, "f32", "bf16", 64, True, "none", False, True), (33, 8224, 40, "bf16", "bf16", 256, True, "silu", True, True),
    (48, 1120, 136, "f32", "f32", 128, True, "silu", True, True), (64, 4096, 1536, "bf16", "bf16", 128, True, "none", True, True),
    (65, 544, 96, "bf16", "bf16", 32, True, "gelu", True, True), (150, 1312, 520, "f32", "f32", 384, True, "none", False, False),
    (20, 16384, 1000, "bf16", "bf16", 16384, True, "none", False, True), (5, 11008, 2048, "f32", "f32", 64, False, "none", False, False),
    (3, 1536, 16384, "bf16", "bf16", 128, True, "none", False, False),
]
# every kind of tiles (rows x columns 1x1, 1x2, 1x4, 2x2, 2x4) with each kind of group
Q4 += [(M, K, N, dtype, "bf16", group, True, "silu", True, True) for dtype in ("bf16", "f32") for group in (32, 64, 256)
       for M, K, N in ((12, 1120, 1000), (12, 1120, 8200), (16, 480, 20008), (40, 480, 4104), (37, 480, 12296), (100, 2208, 9000))]


@pytest.mark.parametrize("case", Q4, ids=lambda c: "%dx%dx%d-%s-s%s-g%d-z%d-%s-b%d-r%d" % c)
def test_4bit(case):
    M, K, N, dtype, st, group, zero, act, bias, res = case
    print("[gpu case] q4", case, flush=True)
    n = maker(M + K + N)
    x, b, r = n((M, K), dtype), n((N,), std=0.2) if bias else None, n((M, N), dtype) if res else None
    q, scale, z, w = weights4(N, K, group, M + N, zero, st)
    got = ms.linear_q4(x, q, scale, z, b, r, group=group, act=ACTS[act])
    close("out", got, finish_ref(mm(x, w), b, act, r), dtype)
    assert torch().equal(got, ms.linear_q4(x, q, scale, z, b, r, group=group, act=ACTS[act]))
    if res:
        buf = r.clone()
        assert ms.linear_q4(x, q, scale, z, b, buf, group=group, act=ACTS[act], out=buf) is buf and torch().equal(buf, got)


def test_4bit_exact_products():
    """Whole numbers and scales of powers of two: every sum is exact, so the layout shows without a tolerance."""
    t = torch()
    gen = t.Generator(device="cpu")
    gen.manual_seed(5)
    for dtype in (t.bfloat16, t.float32):
        for M, K, N, group in ((1, 256, 40, 32), (16, 160, 24, 64), (17, 1120, 72, 128), (40, 96, 136, 32), (70, 2080, 40, 256)):
            x = t.randint(-2, 3, (M, K), generator=gen).to("cuda:0")
            q = t.randint(0, 16, (N, K), generator=gen).to("cuda:0")
            G = -(-K // group)
            z = t.randint(0, 128, (N, G), generator=gen).to("cuda:0")
            scale = 2.0 ** t.randint(-2, 3, (N, G), generator=gen).float().to("cuda:0")
            at = t.arange(K, device="cuda:0") // group
            w = (q.double() - z.double()[:, at]) * scale.double()[:, at]
            packed = (q[:, 0::2] | (q[:, 1::2] << 4)).to(t.uint8)
            got = ms.linear_q4(x.to(dtype), packed, scale.to(dtype), z.to(t.uint8), group=group)
            assert t.equal(got, mm(x, w).float().to(dtype)), (dtype, M, K, N, group)


@pytest.mark.parametrize("M", [4, 60])
def test_4bit_rows_stay_apart(M):
    n = maker(M)
    x = n((M, 160), "bf16")
    q, scale, z, w = weights4(40, 160, 64, 1, True)
    x[1, 5] = float("nan")
    x[M - 1, 159] = float("inf")
    got = ms.linear_q4(x, q, scale, z, group=64)
    assert bool(got[1].isnan().all()) and bool(got[M - 1].isnan().all())
    good = [m for m in range(M) if m not in (1, M - 1)]
    close("rows", got[good], mm(x[good], w), "bf16")


def test_4bit_values_of_every_size():
    """Rows of 2^±100: nothing on the way passes the range of float32."""
    t = torch()
    n = maker(1)
    for dtype in ("bf16", "f32"):
        x = n((3, 256), dtype)
        x[1] *= 2.0 ** 100
        x[2] *= 2.0 ** -90
        q, scale, z, w = weights4(24, 256, 64, 1, True)
        got = ms.linear_q4(x, q, scale, z, group=64)
        want = mm(x, w)
        for m in range(3):
            close("row %d" % m, got[m], want[m], dtype)


def test_other_stream_and_graph():
    t = torch()
    for M in (6, 100):
        n = maker(M)
        x, sx = rows8(n((M, 4096)))
        w, sw = rows8(n((264, 4096)))
        y, r = n((M, 1056), "bf16"), n((M, 264), "bf16")
        q, scale, z, _ = weights4(264, 1056, 32, 1, True)

        def both(**kw):
            return [ms.linear_q8(x, sx, w, sw, None, r, act=ms.ACT_SILU, **kw),
                    ms.linear_q4(y, q, scale, z, None, r, group=32, act=ms.ACT_SILU, **kw)]

        want = both()
        t.cuda.synchronize()
        s = t.cuda.Stream()
        got = both(stream=s)
        s.synchronize()
        assert all(t.equal(a, b) for a, b in zip(got, want))
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            got = both()
        for k in range(3):
            for v in got:
                v.zero_()
            r.copy_(n((M, 264), "bf16"))
            y.copy_(n((M, 1056), "bf16"))
            graph.replay()
            t.cuda.synchronize()
            junk = t.randn(1 << 20, device="cuda:0").sum().item()
            assert junk == junk
            assert all(t.equal(a, b) for a, b in zip(got, both())), k


def test_more_elements_than_32_bits_count():
    t = torch()
    M, K, N = 270000, 32, 8192
    print("[gpu case] q8 sizes", M, K, N, flush=True)
    n = maker(4)
    x, sx = rows8(n((256, K)))
    w, sw = rows8(n((N, K)))
    X, SX = x.view(t.uint8).repeat(M // 256 + 1, 1)[:M].contiguous().view(t.float8_e4m3fn), sx.repeat(M // 256 + 1)[:M].contiguous()
    got, want = ms.linear_q8(X, SX, w, sw), ms.linear_q8(x, sx, w, sw)
    tail = M % 256
    assert t.equal(got[-tail:], want[:tail]) and t.equal(got[:256], want)


def test_binding_refusals():
    t = torch()
    z = lambda *s, dtype=t.float32: t.zeros(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    e = t.float8_e4m3fn
    x, sx, w, sw = z(4, 64, dtype=e), z(4), z(32, 64, dtype=e), z(32)
    for bad in ((x, sx, z(32, 48, dtype=e), sw), (x, z(5), w, sw), (x, sx, w, z(31)), (x, sx, w, sw, z(31)),
                (x, sx, w, sw, None, z(4, 31))):
        with pytest.raises(ValueError):
            ms.linear_q8(*bad)
    for bad in ((z(4, 64), sx, w, sw), (x, sx, z(32, 64), sw), (x, sx.bfloat16(), w, sw), (x.view(t.uint8), sx, w, sw),
                (x, sx, w, sw, None, z(4, 32, dtype=t.float16))):
        with pytest.raises(TypeError):
            ms.linear_q8(*bad)
    with pytest.raises(TypeError):
        ms.linear_q8(x, sx, w, sw, residual=z(4, 32), dtype=t.bfloat16)
    with pytest.raises(TypeError):
        ms.linear_q8(x, sx, w, sw, dtype=t.float16)
    with pytest.raises(ms.MambaError):
        ms.linear_q8(z(4, 72, dtype=e), sx, z(32, 72, dtype=e), sw)
    with pytest.raises(ms.MambaError):
        ms.linear_q8(x[:0], sx[:0], w, sw)
    y, q, s = z(4, 64), z(32, 32, dtype=t.uint8), z(32, 1)
    for bad in (dict(group=32), dict(group=0), dict(residual=z(4, 31)), dict(bias=z(31)), dict(zero=z(32, 2, dtype=t.uint8))):
        with pytest.raises(ValueError):
            ms.linear_q4(y, q, s, **bad)
    for bad in (dict(zero=z(32, 1)), dict(residual=z(4, 32, dtype=t.bfloat16))):
        with pytest.raises(TypeError):
            ms.linear_q4(y, q, s, **bad)
    with pytest.raises(TypeError):
        ms.linear_q4(y, q.to(t.int8), s)
    with pytest.raises(TypeError):
        ms.linear_q4(y, q, s.half())
    with pytest.raises(ms.MambaError):
        ms.linear_q4(y, q, s, group=96)
    with pytest.raises(ms.MambaError):
        ms.linear_q4(z(4, 48), z(32, 24, dtype=t.uint8), s)
    with pytest.raises(ms.MambaError):
        ms.linear_q4(y[:0], q, s)

"""GPU: how the product of 8-bit operands adds where its outputs are bfloat16 and
its rows are not few.  The 8-bit matrix instructions take eight neighbouring
products at a time and cut each off, towards zero, at 2^-13 of the largest of the
eight (an element below 2^-6 counting as 2^-6, a product of zero not at all); the
sums of eights are added in float32.  So each of the seven others loses less than 2^-13 of the
largest, and the rest is float32: at most K/8 joins, each off by at most 2^-23
of what has been added, two roundings' worth (instructions that cut off
included).  A bias of less the exact sum takes the sum away again, so that the
bfloat16 output shows the error itself to 2^-8 of it."""
import pytest

import selective_state_space_mamba_amd as ms

from ffutil import planned_kind
from scanutil import torch

pytestmark = pytest.mark.gpu

# Sizes of each kernel: few rows in blocks of 16, 32 and 64, the long tile with four and eight stages, each tile whole and
# in shares of the contraction (False, True).
KINDS = {(8, 1040, 72): ("rows", 1), (241, 544, 296): ("rows", 2), (215, 560, 584): ("rows", 4), (300, 528, 64): ("long", 4),
         (1000, 4112, 200): ("long", 8), (300, 144, 64): ("tile", 128, 128, False), (300, 8208, 264): ("tile", 128, 128, True),
         (5428, 528, 1440): ("tile", 256, 192, False), (7097, 7008, 528): ("tile", 256, 192, True),
         (2000, 144, 6152): ("tile", 256, 256, False), (6979, 8656, 584): ("tile", 256, 256, True)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


def e4m3(v):
    return v.clamp(-448, 448).to(torch().float8_e4m3fn)


def product(x, w, M, bias, dtype=None):
    """x [R][K] repeated to M rows, w [N][K], both e4m3; scales of one."""
    t = torch()
    rows = x.view(t.uint8).repeat(-(-M // x.shape[0]), 1)[:M].contiguous().view(x.dtype)
    one = t.ones(max(M, w.shape[0]), device="cuda:0")
    return ms.linear_q8(rows, one[:M].contiguous(), w, one[:w.shape[0]].contiguous(), bias, dtype=dtype)


def sums(x, w):
    """Of one row x [K] and w [N][K]: the exact sum, the magnitudes' sum, and the eights' largest products added."""
    t = torch()
    a, b = x.double(), w.double()
    p = a * b
    least = lambda v: v.abs().clamp(min=2.0 ** -6) * (v != 0)  # noqa: E731
    top = (least(a) * least(b)).view(w.shape[0], -1, 8).amax(2).sum(1)
    return p.sum(1), p.abs().sum(1), top


def check(name, x, w, M):
    """Every column against the bound; every row of equal inputs the same.  Returns the mean error over the magnitudes' sum."""
    t = torch()
    exact, size, top = sums(x[0], w)
    bias = (-exact).float()
    got = product(x, w, M, bias)
    assert got.dtype is t.bfloat16 and t.equal(got, got[:1].expand(M, -1))
    err = got[0].double() - (exact + bias.double())
    tol = (7 * 2.0 ** -13 * top + x.shape[1] / 8 * 2.0 ** -23 * size) * (1 + 2.0 ** -8)
    print("%s: worst %.3f of the bound, mean %.2e of the magnitudes" % (name, float((err.abs() / tol).max()), float((err / size).mean())),
          flush=True)
    assert bool((err.abs() <= tol).all()), name
    return float((err / size).mean())


@pytest.mark.parametrize("size", KINDS, ids=lambda s: "%dx%dx%d" % s)
def test_bound_in_every_kernel(size):
    """Values of random signs, of one sign, and spread over the range of e4m3 with its subnormals."""
    t = torch()
    M, K, N = size
    kind = planned_kind("q8", M, K, N)
    print("[gpu case] q8 sums", size, kind, flush=True)
    assert KINDS[size] == (kind[:3] + (kind[3] > 1,) if kind[0] == "tile" else kind)
    g = t.Generator(device="cuda:0")
    g.manual_seed(M + K + N)
    n = lambda *s: t.randn(*s, generator=g, device="cuda:0")  # noqa: E731
    check("normal", e4m3(n(1, K)), e4m3(n(N, K)), M)
    check("positive", e4m3(n(1, K).abs()), e4m3(n(N, K).abs()), M)
    check("wide", e4m3(t.exp(2 * n(1, K))), e4m3(t.exp(2 * n(N, K))), M)
    check("wide, both signs", e4m3(t.exp(2 * n(1, K)) * n(1, K).sign()), e4m3(t.exp(2 * n(N, K))), M)
    check("small", e4m3(n(1, K) * 2.0 ** -6), e4m3(n(N, K) * 2.0 ** -6), M)


@pytest.mark.parametrize("M", [8, 200])
def test_long_positive_sums(M):
    """What is lost does not depend on how many eights are added: up to 65536 elements of one sign."""
    t = torch()
    for K in (1024, 8192, 65536):
        g = t.Generator(device="cuda:0")
        g.manual_seed(K)
        n = lambda *s: t.randn(*s, generator=g, device="cuda:0")  # noqa: E731
        x, w = e4m3(t.exp(2 * n(1, K))), e4m3(t.exp(2 * n(64, K)))
        print("[gpu case] q8 positive", M, K, planned_kind("q8", M, K, 64), flush=True)
        mean = check("K %d" % K, x, w, M)
        assert -7 * 2.0 ** -13 < mean < 7 * 2.0 ** -13


@pytest.mark.parametrize("M,K,N", [(1, 4096, 200), (8, 65536, 72), (40, 1040, 72), (241, 544, 296), (215, 560, 584)])
def test_few_rows_add_in_float32(M, K, N):
    """Also for bfloat16 outputs: nothing is cut off."""
    t = torch()
    assert planned_kind("q8", M, K, N)[0] == "rows"
    g = t.Generator(device="cuda:0")
    g.manual_seed(K)
    n = lambda *s: t.randn(*s, generator=g, device="cuda:0")  # noqa: E731
    x, w = e4m3(t.exp(2 * n(1, K))), e4m3(t.exp(2 * n(N, K)))
    exact, size, _ = sums(x[0], w)
    bias = (-exact).float()
    got = product(x, w, M, bias)
    err = got[0].double() - (exact + bias.double())
    print("M %d K %d: worst %.2e, mean %.2e" % (M, K, float((err.abs() / size).max()), float((err / size).mean())), flush=True)
    assert got.dtype is t.bfloat16 and t.equal(got, got[:1].expand(M, -1))
    # (32 products and the sum so far an instruction, 8 waves' joins, roundings of 2^-24 of the magnitudes, twice)
    assert bool((err.abs() <= (K / 32 + 8) * 2.0 ** -23 * size).all())


def test_float32_outputs_add_in_float32():
    """The same sums asked for in float32: nothing is cut off."""
    t = torch()
    for M, K in ((8, 4096), (300, 4096), (300, 8208), (20000, 1040)):
        g = t.Generator(device="cuda:0")
        g.manual_seed(K)
        n = lambda *s: t.randn(*s, generator=g, device="cuda:0")  # noqa: E731
        x, w = e4m3(t.exp(2 * n(1, K))), e4m3(t.exp(2 * n(64, K)))
        exact, size, _ = sums(x[0], w)
        bias = (-exact).float()
        err = product(x, w, M, bias, t.float32)[0].double() - (exact + bias.double())
        print("M %d K %d: worst %.2e" % (M, K, float((err.abs() / size).max())), flush=True)
        assert bool((err.abs() <= K / 8 * 2.0 ** -23 * size).all()), (M, K)


@pytest.mark.parametrize("size", KINDS, ids=lambda s: "%dx%dx%d" % s)
def test_products_of_like_size_are_exact(size):
    """Elements of 1 to 15: products between 2^0 and 2^8, whose last bits, 2^-6, lie above 2^-13 of the largest one's
    2^6.  Sums of 1024 of them are exact in float32 (64·225·1024 < 2^24), and zeros take up the rest of K."""
    t = torch()
    M, K, N = size
    g = t.Generator(device="cuda:0")
    g.manual_seed(K)

    def values(*s):
        v = (1 + t.randint(0, 8, s, generator=g, device="cuda:0") / 8) * 2.0 ** t.randint(0, 4, s, generator=g, device="cuda:0")
        return v * (1 - 2 * t.randint(0, 2, s, generator=g, device="cuda:0"))

    x, w = values(3, K), values(N, K)
    x[:, t.randperm(K, generator=g, device="cuda:0")[1024:]] = 0
    x, w = e4m3(x), e4m3(w)
    exact = sums(x[0], w)[0]
    got = product(x[:1], w, M, -exact.float())
    assert bool((got == 0).all())
    got = product(x, w, M, None)
    want = t.matmul(x.double(), w.double().t().contiguous()).float().bfloat16()
    assert t.equal(got, want.repeat(-(-M // 3), 1)[:M])


@pytest.mark.parametrize("M", [5, 60, 254, 1000, 20000])
def test_every_pair_of_codes(M):
    """A diagonal weight of every finite code under rows of every finite code: one product a sum, eight bits, exact in
    bfloat16.  (512 rows and columns: few rows, the long tile and the others.)"""
    t = torch()
    codes = t.arange(256, dtype=t.uint8, device="cuda:0")
    codes = codes[(codes & 127) != 127]
    k = t.arange(512, device="cuda:0")
    x = codes[(t.arange(M, device="cuda:0")[:, None] + k * 37) % 254].view(t.float8_e4m3fn)
    w = t.zeros(512, 512, dtype=t.uint8, device="cuda:0")
    w[k, k] = codes[k % 254]
    w = w.view(t.float8_e4m3fn)
    one = t.ones(max(M, 512), device="cuda:0")
    got = ms.linear_q8(x, one[:M].contiguous(), w, one[:512].contiguous())
    want = x.double() * codes[k % 254].view(t.float8_e4m3fn).double()
    print("[gpu case] q8 codes", M, planned_kind("q8", M, 512, 512), flush=True)
    assert got.dtype is t.bfloat16 and bool((got.double() == want).all())

"""GPU: every tile, operand layout and sharing of the matrix product (the sizes
of linear_tiles, which a test on the host holds to that) with whole numbers, so
small that every sum is exact in float32: the results have to be equal to the
float64 product's, rounded once, and to themselves on every call."""
import pytest

import selective_state_space_mamba_amd as ms

from linear_tiles import CASES, DW, DX, FWD, sizes
from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%s-%dx%dx%d" % ((("fwd", "dx", "dw")[c[0]],) + c[1:4]))
def test_exact_products(case):
    t = torch()
    product, m, n, k = case[:4]
    M, K, N = sizes(product, m, n, k)
    print("[gpu case] linear tile", case, flush=True)
    g = t.Generator(device="cuda:0")
    g.manual_seed(m + n + k + product)

    def whole(lo, hi, *shape, dtype=t.bfloat16):
        return t.randint(lo, hi + 1, shape, generator=g, device="cuda:0").to(dtype)

    x, w, dout = whole(-2, 2, M, K), whole(-1, 1, N, K), whole(-1, 1, M, N)
    b, res = whole(-5, 5, N, dtype=t.float32), whole(-9, 9, M, N)
    if product == FWD:
        def call():
            return ms.linear_fwd(x, w, b, res, act=ms.ACT_RELU, want_pre=True)
        pre = t.matmul(x.double(), w.double().t().contiguous()) + b.double()
        want = (pre.clamp(min=0) + res.double()).float().bfloat16(), pre.float()
    elif product == DX:
        def call():
            return (ms.linear_bwd(x, w, dout=dout, want_dweight=False, want_dbias=False)["dx"],)
        want = (t.matmul(dout.double(), w.double()).float().bfloat16(),)
    else:
        assert product == DW
        def call():
            return (ms.linear_bwd(x, w, dout=dout, want_dx=False, want_dbias=False)["dweight"],)
        want = (t.matmul(dout.double().t().contiguous(), x.double()).float().bfloat16(),)
    for _ in range(4):
        for got, exp in zip(call(), want):
            assert t.equal(got, exp)

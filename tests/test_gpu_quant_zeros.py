"""GPU: the product with 4-bit weights takes every byte as a zero point, not only
those of 4 or 7 bits."""
import pytest

import selective_state_space_mamba_amd as ms

from ffutil import close, dtype_of, maker, mm
from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


def make(N, K, group, seed, scale_type):
    """Every byte among the zeros; packed weights, scale, zero and what they stand for."""
    t = torch()
    g = t.Generator(device="cpu")
    g.manual_seed(seed)
    G = -(-K // group)
    q = t.randint(0, 16, (N, K), generator=g)
    z = (t.arange(N * G).view(N, G) * 37 + 128) % 256
    scale = (2.0 ** t.randint(-2, 3, (N, G), generator=g)).to(scale_type)
    at = t.arange(K) // group
    w = (q.double() - z.double()[:, at]) * scale.double()[:, at]
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).to(t.uint8)
    return [v.to("cuda:0") for v in (packed, scale, z.to(t.uint8), w)]


SIZES = [(1, 256, 40, 32), (16, 160, 264, 64), (17, 1120, 72, 128), (40, 96, 1000, 32), (70, 2080, 40, 256), (100, 480, 12296, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "%dx%dx%d-g%d" % s)
def test_every_zero(size, dtype):
    """Whole numbers and scales of powers of two: every sum is exact in float32 (of terms up to 2·255·4 in
    quarters, whose signs are random: far below 2^24 of them), the bfloat16 rows' of 1 + q/128 too."""
    M, K, N, group = size
    t = torch()
    g = t.Generator(device="cpu")
    g.manual_seed(M)
    x = t.randint(-2, 3, (M, K), generator=g).to("cuda:0")
    packed, scale, z, w = make(N, K, group, K, dtype_of(dtype))
    assert N * -(-K // group) < 128 or int(z.max()) > 250
    got = ms.linear_q4(x.to(dtype_of(dtype)), packed, scale, z, group=group)
    assert t.equal(got, mm(x, w).float().to(dtype_of(dtype)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_zero_on_values(dtype):
    """Rows of normal values; tolerances as for zeros of 4 bits, of larger weights."""
    n = maker(3)
    x = n((9, 512), dtype)
    packed, scale, z, w = make(200, 512, 64, 5, dtype_of("f32"))
    close("out", ms.linear_q4(x, packed, scale, z, group=64), mm(x, w), dtype)

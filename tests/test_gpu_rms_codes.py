"""GPU: the codes of the norm's 8-bit output, bit for bit: the float32 quotient
y / scale rounded to nearest even, next to every border between two codes, and
scale the float32 quotient of the row's largest by 448."""
import pytest

import selective_state_space_mamba_amd as ms

from ffutil import maker
from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


def codes(y, scale):
    """On the CPU, whose division and conversion are the types' own."""
    t = torch()
    return (y.cpu() / scale.cpu()).to(t.float8_e4m3fn).view(t.uint8)


def borders(scale):
    """Values within 3 float32 steps of every border between two codes, times scale."""
    t = torch()
    v = t.arange(127, dtype=t.uint8).view(t.float8_e4m3fn).float()
    mid = ((v[1:] + v[:-1]) / 2 * scale).view(t.int32)
    return t.cat([(mid + k).view(t.float32) for k in range(-3, 4)])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_beside_every_border(dtype):
    """Rows of ones have rstd 1 (eps 0), so that y is the weight itself."""
    t = torch()
    g = t.Generator(device="cpu")
    g.manual_seed(1)
    other = 0
    for k in range(60):
        top = (1 + t.rand(1, generator=g)) * 2.0 ** int(t.randint(-20, 20, (1,), generator=g))
        scale = top / 448
        y = t.cat([top, borders(scale), -borders(scale)])
        y = y[y.abs() <= top]
        other += int((codes(y, scale) != (y * (1 / scale)).to(t.float8_e4m3fn).view(t.uint8)).sum())
        x = t.ones(3, y.numel(), dtype=t.float32 if dtype == "f32" else t.bfloat16, device="cuda:0")
        q, got, _ = ms.rms_norm_q8(x, y.to("cuda:0"), eps=0.0)
        assert t.equal(got.cpu(), scale.expand(3)), k
        assert t.equal(q.cpu().view(t.uint8), codes(y, scale).expand(3, -1)), k
    print("borders where the reciprocal's product has another code: %d" % other, flush=True)
    assert other > 50


@pytest.mark.parametrize("M,D", [(3000, 64), (500, 301), (40, 1536), (700, 1536), (2000, 2048), (9, 5000), (5, 16384)])
def test_codes_of_rows(M, D):
    """Of the normalised rows that the float32 form returns, whose arithmetic is the same."""
    t = torch()
    n = maker(M)
    x, w = n((M, D)), n((D,))
    x[0] = 0  # (and -0 where the weight is negative)
    x[1] *= 1e-30
    y, _, _ = ms.rms_norm_fwd(x, w, eps=1e-12)
    q, scale, _ = ms.rms_norm_q8(x, w, eps=1e-12)
    top = (y.cpu().abs().amax(1) / 448).clamp(min=2.0 ** -100)
    assert t.equal(scale.cpu(), top)
    assert t.equal(q.cpu().view(t.uint8), codes(y, scale[:, None]))


@pytest.mark.parametrize("D", [64, 300, 1536, 5000])
def test_codes_of_an_infinite_row(D):
    """An infinite y makes the scale infinite: the others' quotients are zeros, its own is NaN."""
    t = torch()
    n = maker(D)
    x, w = n((3, D)), n((D,))
    w[5] = float("inf")
    q, scale, _ = ms.rms_norm_q8(x, w, eps=1e-5)
    y, _, _ = ms.rms_norm_fwd(x, w, eps=1e-5)
    want = codes(y, scale[:, None]).view(t.float8_e4m3fn).float()
    assert bool(scale.isinf().all())
    got = q.cpu().float()
    assert t.equal(got.isnan(), want.isnan()) and t.equal(got.nan_to_num(), want.nan_to_num())
    assert bool((got.isnan().sum(1) == 1).all()) and bool((got[:, :5] == 0).all())

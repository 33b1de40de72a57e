"""GPU: sums of one sign in the gated pair of float32, whose tiles multiply three
bfloat16 terms of each element.  Rounding to nearest errs to either side: over
the outputs of a product its mean is near zero, however long the contraction.
What the terms leave out, and small products that vanish in a large sum, would
err to one side and show in the mean."""
import pytest

import selective_state_space_mamba_amd as ms

from ffutil import mm
from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


def compare(name, got, want, K):
    """Each sum of 16 products is joined by two additions, each off by at most 2^-24 of the sum so far (whose terms are
    of one sign), and the shares' and rows' joins are a few more: their mean over the outputs within 4 roots of their
    number, over as many roots of the outputs, of 2^-24.  Outputs share their rows and columns, and roundings repeat
    where the sums do: ten times that, and 2^-29 (a thirtieth of a rounding) at least.  The largest: all roundings on
    one side would be (K/8 + 16)·2^-24; as errors of either sign 8 roots of as many."""
    err = (got.double() - want) / want
    steps = K / 8 + 16
    mean_tol = max(10 * 4 * (steps / err.numel()) ** 0.5 * 2.0 ** -24, 2.0 ** -29)
    top_tol = 8 * steps ** 0.5 * 2.0 ** -24
    mean, top = float(err.mean()), float(err.abs().max())
    print("%s: mean %.2e of %.2e, largest %.2e of %.2e" % (name, mean, mean_tol, top, top_tol), flush=True)
    assert abs(mean) <= mean_tol and top <= top_tol, (name, mean, top)


@pytest.mark.parametrize("size", [(129, 72, 136), (300, 2056, 264), (1037, 520, 1384), (100, 1024, 1024), (2048, 4096, 768),
                                  (768, 512, 4096), (4100, 264, 520)], ids=lambda s: "%dx%dx%d" % s)
def test_mean_error_of_positive_sums(size):
    """x, the weights and dout between 1 and 2; pre of ones makes dg and du of act none dout itself."""
    t = torch()
    M, K, N = size
    print("[gpu case] gated sums", size, flush=True)
    g = t.Generator(device="cuda:0")
    g.manual_seed(M)
    u = lambda *s: 1 + t.rand(*s, generator=g, device="cuda:0")  # noqa: E731
    x, wg, wu, dout = u(M, K), u(N, K), u(N, K), u(M, N)
    _, pre = ms.gated_linear_fwd(x, wg, wu, act=ms.ACT_NONE, want_pre=True)
    compare("gate", pre[0], mm(x, wg), K)
    compare("up", pre[1], mm(x, wu), K)
    got = ms.gated_linear_bwd(x, wg, wu, dout=dout, pre=t.ones_like(pre), act=ms.ACT_NONE)
    compare("dx", got["dx"], t.matmul(dout.double(), wg.double() + wu.double()), 2 * N)
    dw = mm(dout.t(), x.t())
    compare("dw_gate", got["dw_gate"], dw, M)
    assert t.equal(got["dw_gate"], got["dw_up"])


def test_every_bit_of_an_element_counts():
    """Elements of 24 significant bits of either sign against a weight of single ones: each output is one element,
    which its three terms give back exactly; up to the largest float32 and down to 2^-100 (whose last bit a term still
    holds)."""
    t = torch()
    g = t.Generator(device="cuda:0")
    g.manual_seed(1)
    M, K = 200, 64
    for e in (-100, -30, 0, 60, 127):
        bits = t.randint(0, 1 << 23, (M, K), generator=g, device="cuda:0", dtype=t.int32) | (e + 127) << 23
        bits[0, :] |= 0x7fffff  # the largest of the exponent, 3.4e38 of the last
        x = bits.view(t.float32) * (1 - 2 * t.randint(0, 2, (M, K), generator=g, device="cuda:0"))
        w = t.eye(K, device="cuda:0")
        _, pre = ms.gated_linear_fwd(x, w, w, act=ms.ACT_NONE, want_pre=True)
        assert t.equal(pre[0], x) and t.equal(pre[1], x), e
        dx = ms.gated_linear_bwd(x, w, w, dout=t.ones(M, K, device="cuda:0"), pre=t.stack([x, t.zeros_like(x)]), act=ms.ACT_NONE,
                                 want_dweight=False, want_dbias=False)["dx"]  # dg = 0, du = x
        assert t.equal(dx, x), e

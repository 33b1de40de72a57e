"""GPU: statistics of maps in which single rows lie far from all others (the
first token of a sequence often does), against float64.

Tolerance, written before the first run.  A group's M = Σ (x - mean)² is a sum
of terms that are not negative, joined from partial sums over at most some
hundred rows of a thread and a tree over the threads: about (100 + 10)·2^-24 =
7e-6 of M if every rounding went the same way, half of that in rstd, and far
less as they do not.  1e-5 of rstd is asked of every group, the float32 bars of
2e-4 (normwise) and 2e-5 (L2) of the outputs and of dx.  A mean is rounded to
2^-24 of the largest value that enters it, once in every block of rows and join:
a hundred times that is asked."""
import pytest

import selective_state_space_mamba_amd as ms

from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield


def near(name, got, want, emax, el2):
    d = (got.double() - want).abs()
    a, b = float(d.max() / want.abs().max()), float(d.norm() / want.norm())
    print("%s: max %.2e l2 %.2e" % (name, a, b), flush=True)
    assert a <= emax and b <= el2, (name, a, b)


@pytest.mark.parametrize("off", [100.0, 1000.0, 10000.0])
@pytest.mark.parametrize("shape", [
    # one workgroup an item: many rows in few channels; rows that end inside a thread's block; many short items
    (2, 2048, 8), (3, 1021, 24), (1500, 300, 48),
    # runs of rows, a workgroup each: two long ones an item, many short ones
    (512, 1200, 64), (1, 4099, 64), (700, 1000, 192),
], ids=lambda s: "%dx%dx%d" % s)
def test_rows_far_from_the_others(shape, off):
    t = torch()
    B, L, D = shape
    print("[gpu case] norm outliers", shape, off, flush=True)
    g = t.Generator(device="cuda:0")
    g.manual_seed(B + L)
    x = t.randn(B, L, D, generator=g, device="cuda:0")
    x[:, 0] += off          # the item's first row, which is a run's first row too
    x[:, L // 2] -= off     # and the second run's where there are two
    dout = t.randn(B, L, D, generator=g, device="cuda:0")
    for G in (1, D):
        out, mean, rstd = ms.group_norm_fwd(x, G)
        got = ms.group_norm_bwd(x, G, dout=dout, mean=mean, rstd=rstd)["dx"]
        v = x.double().view(B, L, G, D // G)
        m = v.mean((1, 3), keepdim=True)
        r = 1 / t.sqrt(((v - m) ** 2).mean((1, 3), keepdim=True) + 1e-5)
        xh = (v - m) * r
        rel = float(((rstd.double() - r.view(B, G)).abs() / r.view(B, G)).max())
        am = float((mean.double() - m.view(B, G)).abs().max())
        print("G %d: rstd %.2e, mean off by %.2e" % (G, rel, am), flush=True)
        assert rel <= 1e-5
        assert am <= 100 * 2.0 ** -24 * off
        near("out", out, xh.reshape(B, L, D), 2e-4, 2e-5)
        dv = dout.double().view(B, L, G, D // G)
        want = r * (dv - dv.mean((1, 3), keepdim=True) - xh * (dv * xh).mean((1, 3), keepdim=True))
        near("dx", got, want.reshape(B, L, D), 2e-4, 2e-5)


def test_a_common_offset_costs_no_bits():
    """Every row 10000 deviations from zero, exactly: the statistics are those of the rows without it."""
    t = torch()
    for B, L, D in ((2, 2048, 8), (2, 5000, 64)):
        g = t.Generator(device="cuda:0")
        g.manual_seed(L)
        x = t.randint(-8, 9, (B, L, D), generator=g, device="cuda:0").float() + 10000.0
        for G in (1, D):
            _, mean, rstd = ms.group_norm_fwd(x, G)
            v = x.double().view(B, L, G, D // G)
            m = v.mean((1, 3), keepdim=True)
            r = 1 / t.sqrt(((v - m) ** 2).mean((1, 3), keepdim=True) + 1e-5)
            assert float(((rstd.double() - r.view(B, G)).abs() / r.view(B, G)).max()) <= 1e-5
            assert float((mean.double() - m.view(B, G)).abs().max()) <= 4 * 2.0 ** -24 * 10000.0

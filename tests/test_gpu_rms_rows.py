"""GPU: the root-mean-square norm over more rows than one axis of a grid has
workgroups for, narrow rows that share a wave, every row of every output.  Rows
of one sign and magnitude have rstd 1 (eps 0) and xh of 1 or -1, and gradients
of small whole numbers keep every sum exact, so nothing needs a tolerance."""
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
    torch().cuda.empty_cache()


# channels (8, 16 and 32 lanes of a wave a row) and rows of a workgroup of 256 threads
@pytest.mark.parametrize("D,per", [(1, 32), (8, 32), (64, 32), (128, 16), (256, 8)])
def test_rows_past_an_axis_of_workgroups(D, per):
    t = torch()
    M = per * (1 << 20) + 5 * per + 3  # (an axis takes 2^20 workgroups)
    print("[gpu case] rms rows", M, D, flush=True)
    g = t.Generator(device="cuda:0")
    g.manual_seed(D)
    ints = lambda lo, hi, *s: t.randint(lo, hi + 1, s, generator=g, device="cuda:0", dtype=t.int8).bfloat16()  # noqa: E731
    sign = 2 * ints(0, 1, M, 1) - 1
    x = sign.expand(M, D).contiguous()
    w = 2.0 ** t.randint(-2, 3, (D,), generator=g, device="cuda:0").float()
    out, _, rstd = ms.rms_norm_fwd(x, w, eps=0.0)
    assert bool((rstd == 1).all())
    assert t.equal(out, sign * w.bfloat16())
    q, scale, _ = ms.rms_norm_q8(x, w, eps=0.0)
    top = w.max() / 448
    assert bool((scale == scale[0]).all()) and abs(float(scale[0] / top) - 1) <= 2.0 ** -23
    assert t.equal(q[:, 0].view(t.uint8) >> 7, (sign[:, 0] < 0).to(t.uint8)) and t.equal(q[sign[:, 0] > 0].view(t.uint8).amin(0),
                                                                                    q[sign[:, 0] > 0].view(t.uint8).amax(0))
    del out, q
    dout, dadded = ints(-1, 1, M, D), ints(-9, 9, M, D)
    got = ms.rms_norm_bwd(x, w, dout=dout, rstd=rstd, dadded=dadded)
    dw = t.zeros(D, dtype=t.float64, device="cuda:0")
    step = (1 << 27) // D
    for a in range(0, M, step):
        b = slice(a, min(M, a + step))
        s, dy = sign[b].float(), dout[b].float()
        dw += (dy * s).sum(0, dtype=t.float64)
        c = (dy * w * s).sum(1, keepdim=True) / D  # (quarters, and a power of two below)
        assert t.equal(got["dx"][b], (dy * w - s * c + dadded[b].float()).bfloat16()), a
    assert float(dw.abs().max()) < 1 << 24 and t.equal(got["dweight"].double(), dw)


def test_weight_gradient_of_many_wide_rows():
    """Rows with a wave or more each: 2^31 elements and more."""
    t = torch()
    for D in (512, 2048, 16384):
        M = (1 << 31) // D + 37
        print("[gpu case] rms dweight", M, D, flush=True)
        g = t.Generator(device="cuda:0")
        g.manual_seed(D)
        sign = t.randint(0, 2, (M, 1), generator=g, device="cuda:0", dtype=t.int8).bfloat16() * 2 - 1
        dout = t.randint(-1, 2, (M, D), generator=g, device="cuda:0", dtype=t.int8).bfloat16()
        x = sign.expand(M, D).contiguous()
        rstd = t.ones(M, device="cuda:0")
        got = ms.rms_norm_bwd(x, t.ones(D, device="cuda:0"), dout=dout, rstd=rstd)
        dw = t.zeros(D, dtype=t.float64, device="cuda:0")
        step = (1 << 27) // D
        for a in range(0, M, step):
            s, dy = sign[a:a + step].float(), dout[a:a + step].float()
            dw += (dy * s).sum(0, dtype=t.float64)
            c = (dy * s).sum(1, keepdim=True) / D
            assert t.equal(got["dx"][a:a + step], (dy - s * c).bfloat16()), (D, a)
        assert t.equal(got["dweight"].double(), dw)

"""GPU: the operators around the scan at counts and sizes that pass what 32 bits
hold: more workgroups than one axis of a grid takes, tensors of more than 2^31
elements.  References in float64 on the GPU.  Tolerances: the projects' bars
(float32 2e-4 of the largest value and 2e-5 in the L2 norm, bfloat16 1e-2 and
3e-3)."""
import pytest

import selective_state_space_mamba_amd as ms

from scanutil import torch

pytestmark = pytest.mark.gpu
TOL = {"f32": (2e-4, 2e-5), "bf16": (1e-2, 3e-3)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


def near(name, got, want, kind):
    d = (got.double() - want).abs()
    a, b = float(d.max() / want.abs().max()), float(d.norm() / want.norm())
    print("%s: max %.2e l2 %.2e" % (name, a, b), flush=True)
    assert a <= TOL[kind][0] and b <= TOL[kind][1], (name, a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_sequences_than_an_axis_of_workgroups(dtype):
    t = torch()
    B, D = (1 << 23) + 5, 4  # of 512 threads each: 2^32 and more
    print("[gpu case] glr sequences", B, dtype, flush=True)
    g = t.Generator(device="cuda:0")
    g.manual_seed(1)
    dt = t.float32 if dtype == "f32" else t.bfloat16
    x, r, dout = (t.randn(B, 1, D, generator=g, device="cuda:0").to(dt) for _ in range(3))
    init = t.randn(B, D, generator=g, device="cuda:0")
    kw = dict(input_rule=ms.GLR_LERP, initial_state=init)
    out, last = ms.glr_fwd(x, r, **kw)
    got = ms.glr_bwd(x, r, dout=dout, **kw)
    t.cuda.synchronize()
    a = t.sigmoid(r.double())
    want = a * init[:, None].double() + (1 - a) * x.double()
    near("out", out, want, dtype)
    near("last", last, want[:, 0], "f32")
    near("dx", got["dx"], dout.double() * (1 - a), dtype)
    near("dinit", got["dinit"], (dout.double() * a)[:, 0], "f32")
    near("dr", got["dr"], dout.double() * a * (1 - a) * (init[:, None].double() - x.double()), dtype)
    step = init.clone()
    near("step", ms.glr_step(step, x[:, 0], r[:, 0], input_rule=ms.GLR_LERP), want[:, 0], dtype)


def test_more_items_than_an_axis_of_workgroups():
    t = torch()
    B, L, D = (1 << 24) + 3, 2, 8  # of 256 threads each
    print("[gpu case] norm items", B, flush=True)
    g = t.Generator(device="cuda:0")
    g.manual_seed(2)
    x, dout = (t.empty(B, L, D, device="cuda:0", dtype=t.bfloat16) for _ in range(2))
    for v in (x, dout):
        v.normal_(generator=g)
    w = t.linspace(0.5, 1.5, D, device="cuda:0")
    out, mean, rstd = ms.group_norm_fwd(x, 1, w)
    dx = ms.group_norm_bwd(x, 1, w, dout=dout, mean=mean, rstd=rstd)["dx"]
    t.cuda.synchronize()
    for lo in range(0, B, 1 << 21):
        s = slice(lo, lo + (1 << 21))
        v, dv = x[s].double(), dout[s].double() * w.double()
        m = v.mean((1, 2), keepdim=True)
        rs = 1 / t.sqrt(((v - m) ** 2).mean((1, 2), keepdim=True) + 1e-5)
        xh = (v - m) * rs
        near("out", out[s], xh * w.double(), "bf16")
        near("dx", dx[s], rs * (dv - dv.mean((1, 2), keepdim=True) - xh * (dv * xh).mean((1, 2), keepdim=True)), "bf16")

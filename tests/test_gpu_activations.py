"""GPU: the activations of the matrix product's and the normalisation's epilogues
against float64.  A product with the identity hands the activation its argument
exactly, in float32, and the gradient's products its derivative.

Tolerances of gelu, u·Φ(u), written before the first run.  Above zero Φ is 1 less
a tail: some six roundings of 2^-24 of it, 4e-7.  Below it is the tail itself,
e^{-u²/2} times a fitted factor: the same roundings, and the exponent's two, up to
2^-24·0.72·u² each in its base: 1e-6 + 1e-7·u².  Over normal arguments the
roundings are independent, about 2^-24/sqrt(3) = 3.4e-8 each, and most
weigh less than whole: 7e-8 of the values, 1e-7 of the derivative."""
import numpy as np
import pytest

import selective_state_space_mamba_amd as ms

from layerutil import ACTS, act_ref, from_dev, to_dev
from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield


def through(u, act):
    """The activation and its derivative at u (float32)."""
    t = torch()
    x = to_dev(np.resize(u, (-(-u.size // 8), 8)).astype(np.float32))
    eye = t.eye(8, device="cuda:0")
    out, pre = ms.linear_fwd(x, eye, act=ACTS[act], want_pre=True)
    assert t.equal(pre, x)
    d = ms.linear_bwd(x, eye, dout=t.ones_like(x), pre=pre, act=ACTS[act])["dx"]
    return from_dev(out).ravel()[:u.size], from_dev(d).ravel()[:u.size]


def test_gelu_over_its_range():
    u = np.linspace(-9.0, 9.0, 40001).astype(np.float32)
    u = u[u != 0]
    print("[gpu case] gelu", flush=True)
    got, _ = through(u, "gelu")
    want = act_ref(u.astype(np.float64), "gelu")[0]
    rel = np.abs(got / want - 1)
    for lo in range(-9, 9):
        m = (u >= lo) & (u < lo + 1)
        print("%d: %.1e" % (lo, rel[m].max()), flush=True)
    ask = np.where(u > 0, 4e-7, 1e-6 + 1e-7 * u.astype(np.float64) ** 2)
    assert np.all(rel <= ask), (u[(rel / ask).argmax()], rel[(rel / ask).argmax()])


def test_gelu_over_normal_arguments():
    u = np.random.Generator(np.random.PCG64(2)).standard_normal(1 << 18).astype(np.float32)
    got, d = through(u, "gelu")
    want, wd = act_ref(u.astype(np.float64), "gelu")
    l2 = np.linalg.norm(got - want) / np.linalg.norm(want), np.linalg.norm(d - wd) / np.linalg.norm(wd)
    print("gelu %.2e derivative %.2e" % l2, flush=True)
    assert l2[0] <= 7e-8 and l2[1] <= 1e-7


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_far_arguments(act):
    """Where the exponentials vanish or overflow: 0 or the argument, derivatives of 0 or 1."""
    u = np.float32([-3e38, -1e20, -1e4, -300.0, -120.0, 120.0, 300.0, 1e4, 1e20, 3e38])
    got, d = through(u, act)
    want, wd = act_ref(u.astype(np.float64), act)
    assert np.allclose(got, want, rtol=1e-6, atol=1e-30) and np.allclose(d, wd, rtol=1e-6, atol=1e-30)

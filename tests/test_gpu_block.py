"""The operators together, as examples/recurrent_block.py uses them: forward
and every gradient of a residual block in float32 against the composition of
the plain float64 forms, the token-by-token path against the whole-sequence one,
and the example's own run.

Tolerances, written before the first run: each operator is held to 2e-4
(normwise) and 2e-5 (L2) in float32; a chain of five keeps within the first and
about five times the second, 1e-4.  The two paths of the example differ by bf16
roundings of the same intermediate values, a few 2^-9 of the largest output."""
import importlib.util
import os

import numpy as np
import pytest

import selective_state_space_mamba_amd as ms

from layerutil import from_dev, glr_grads, glr_ref, linear_ref, norm_ref, to_dev
from scanutil import errors, torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    spec = importlib.util.spec_from_file_location("recurrent_block", os.path.join(ROOT, "examples", "recurrent_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def close(name, got, want):
    got, want = from_dev(got), np.asarray(want, np.float64)
    assert got.shape == want.shape and np.all(np.isfinite(got)), name
    emax, el2 = errors(got, want)
    print("%s: max %.2e l2 %.2e" % (name, emax, el2), flush=True)
    assert emax <= 2e-4 and el2 <= 1e-4, (name, emax, el2)


def test_block_forward_and_gradients(example):
    B, L, D, inner, G = 2, 150, 72, 136, 3
    blk = example.RecurrentBlock(D, inner, G, dtype=torch().float32, seed=3)
    r = np.random.Generator(np.random.PCG64(5))
    x, dy = r.standard_normal((2, B, L, D)).astype(np.float32)
    init = r.standard_normal((B, inner)).astype(np.float32)
    reset = (r.uniform(size=(B, L)) < 0.02).astype(np.uint8)
    for k in blk.w:  # biases and norm weights that matter
        if k.startswith("b_") or k.startswith("norm"):
            blk.w[k] = blk.w[k] + to_dev(0.2 * r.standard_normal(tuple(blk.w[k].shape)).astype(np.float32))
    w = {k: from_dev(v) for k, v in blk.w.items()}
    y, last = blk.forward(to_dev(x), to_dev(init), to_dev(reset))
    dx, grads = blk.backward(to_dev(dy))
    # the composition in float64
    x8, dy8 = x.astype(np.float64), dy.astype(np.float64)
    flat = x8.reshape(B * L, 1, D)
    n = norm_ref(flat, G, w["norm_w"], w["norm_b"], "none", 1e-5)[0].reshape(B * L, D)
    g = {k: linear_ref(n, w["w_" + k], w["b_" + k], None, "none")[0].reshape(B, L, inner) for k in example.GATES}
    kw = dict(init=init.astype(np.float64), reset=reset)
    h, want_last, _, _ = glr_ref(g["p"], g["r"], g["i"], g["z"], w["lam"], **kw)
    out, _, go = linear_ref(h.reshape(-1, inner), w["w_o"], w["b_o"], x8.reshape(-1, D), "none", dy8.reshape(-1, D))
    close("y", y, out.reshape(B, L, D))
    close("last_state", last, want_last)
    gr = glr_grads(g["p"], g["r"], g["i"], g["z"], w["lam"], go["dx"].reshape(B, L, inner), **kw)
    want = dict(w_o=go["dweight"], b_o=go["dbias"], lam=gr["dlam"])
    dn = 0.0
    for k, name in zip(example.GATES, ("dx", "dr", "di", "dz")):
        one = linear_ref(n, w["w_" + k], w["b_" + k], None, "none", gr[name].reshape(-1, inner))[2]
        want["w_" + k], want["b_" + k] = one["dweight"], one["dbias"]
        dn = dn + one["dx"]
    norm = norm_ref(flat, G, w["norm_w"], w["norm_b"], "none", 1e-5, dn.reshape(B * L, 1, D))[3]
    want.update(norm_w=norm["dweight"], norm_b=norm["dbias"])
    close("dx", dx, norm["dx"].reshape(B, L, D) + dy8)
    assert sorted(grads) == sorted(want)
    for k in grads:
        close("d" + k, grads[k], want[k])


def test_block_step_by_step(example):
    B, L, D = 3, 70, 72
    blk = example.RecurrentBlock(D, 136, 3, dtype=torch().float32, seed=4)
    x = to_dev(np.random.Generator(np.random.PCG64(6)).standard_normal((B, L, D)).astype(np.float32))
    y, last = blk.forward(x)
    state = torch().zeros_like(last)
    got = torch().stack([blk.step(x[:, t].contiguous(), state) for t in range(L)], 1)
    close("tokens", got, from_dev(y))
    close("state", state, from_dev(last))


def test_example_learns(example):
    losses, off = example.main(steps=40)
    assert losses[-1] < 0.7 * losses[0]  # the toy task is learnable: its loss falls
    assert off < 2e-2

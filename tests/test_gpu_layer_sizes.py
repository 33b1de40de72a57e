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


def test_recurrence_past_2_31_elements():
    """Each way of running (tiles chained; walked), the last item judged at its end: with decays of at most
    sigmoid(2) = 0.88 a window of 512 tokens keeps 1e-28 of what came before it."""
    t = torch()
    for B, L, D in ((1, (1 << 21) + 77, 1028), (2080, 16200, 64)):
        print("[gpu case] glr long", B, L, D, flush=True)
        g = t.Generator(device="cuda:0")
        g.manual_seed(3)
        x, r = (t.empty(B, L, D, dtype=t.bfloat16, device="cuda:0") for _ in range(2))
        x.normal_(generator=g)
        r.normal_(generator=g).clamp_(-2, 2)
        assert x.numel() > 1 << 31
        out, last, saved = ms.glr_fwd_save(x, r, input_rule=ms.GLR_LERP)
        dout = t.zeros_like(x)
        n = 512
        dout[:, -n:].normal_(generator=g)
        grads = ms.glr_bwd(x, r, dout=dout, saved=saved, input_rule=ms.GLR_LERP)
        t.cuda.synchronize()
        del saved
        items = slice(B - 1, B)
        a = t.sigmoid(r[items, -2 * n:].double())
        b = (1 - a) * x[items, -2 * n:].double()
        h, hs, hp = t.zeros(1, D, dtype=t.double, device="cuda:0"), [], []
        for k in range(2 * n):
            hp.append(h)
            h = a[:, k] * h + b[:, k]
            hs.append(h)
        near("out", out[items, -n:], t.stack(hs[n:], 1), "bf16")
        near("last", last[items], h, "f32")
        m, dx, dr = t.zeros_like(h), [], []
        for k in range(2 * n - 1, n - 1, -1):
            m = m + dout[items, k - 2 * n].double()
            dx.append(m * (1 - a[:, k]))
            dr.append(m * a[:, k] * (1 - a[:, k]) * (hp[k] - x[items, k - 2 * n].double()))
            m = m * a[:, k]
        near("dx", grads["dx"][items, -n:], t.stack(dx[::-1], 1), "bf16")
        near("dr", grads["dr"][items, -n:], t.stack(dr[::-1], 1), "bf16")
        assert not bool(grads["dx"][:, :-3 * n].abs().max() > 1e-6)
        del x, r, out, dout, grads


def test_norm_past_2_31_elements():
    t = torch()
    for B, L, D, G in ((1, (1 << 21) + 5, 1032, 3), (4200000, 1, 520, 5), (262147, 1, 8192, 1)):
        print("[gpu case] norm large", B, L, D, G, flush=True)
        g = t.Generator(device="cuda:0")
        g.manual_seed(4)
        x = t.empty(B, L, D, dtype=t.bfloat16, device="cuda:0").normal_(generator=g)
        assert x.numel() > 1 << 31
        out, mean, rstd = ms.group_norm_fwd(x, G)
        dx = ms.group_norm_bwd(x, G, dout=x, mean=mean, rstd=rstd)["dx"]
        t.cuda.synchronize()
        item = B - 1
        v = x[item].double().view(L, G, D // G)
        m, va = v.mean((0, 2), keepdim=True), v.var((0, 2), unbiased=False, keepdim=True)
        rs = 1 / t.sqrt(va + 1e-5)
        xh = (v - m) * rs
        near("mean", mean[item] + 1, m.flatten() + 1, "f32")
        near("rstd", rstd[item], rs.flatten(), "f32")
        near("out", out[item][-1000:], xh.reshape(L, D)[-1000:], "bf16")
        # dout = x: what is left of dx is rstd²·eps·xh, so it is held to the size of its terms
        want = rs * (v - v.mean((0, 2), keepdim=True) - xh * (v * xh).mean((0, 2), keepdim=True))
        assert float((dx[item].double().view(L, G, D // G) - want).abs().max()) <= 1e-4
        del x, out, dx


def test_product_past_2_31_elements():
    t = torch()
    M, K, N = (1 << 21) + 3, 64, 1032
    print("[gpu case] linear large", M, K, N, flush=True)
    g = t.Generator(device="cuda:0")
    g.manual_seed(5)
    x = t.empty(M, K, dtype=t.bfloat16, device="cuda:0").normal_(generator=g)
    w = (t.randn(N, K, generator=g, device="cuda:0") / 8).bfloat16()
    b = t.randn(N, generator=g, device="cuda:0")
    out, pre = ms.linear_fwd(x, w, b, act=ms.ACT_SILU, want_pre=True)
    dout = t.empty(M, N, dtype=t.bfloat16, device="cuda:0").normal_(generator=g)
    assert out.numel() > 1 << 31
    got = ms.linear_bwd(x, w, dout=dout, pre=pre, act=ms.ACT_SILU)
    t.cuda.synchronize()
    rows = slice(M - 500, M)
    u = t.matmul(x[rows].double(), w.double().t().contiguous()) + b.double()
    q = t.sigmoid(u)
    near("pre", pre[rows], u, "f32")
    near("out", out[rows], u * q, "bf16")
    dp = dout[rows].double() * q * (1 + u * (1 - q))
    want = t.matmul(dp, w.double())
    d = (got["dx"][rows].double() - want)
    assert float(d.norm() / want.norm()) <= 4e-3  # (one rounding more, of dP)
    dw, db = t.zeros(N, K, dtype=t.double, device="cuda:0"), t.zeros(N, dtype=t.double, device="cuda:0")
    for lo in range(0, M, 1 << 17):
        s = slice(lo, lo + (1 << 17))
        u = pre[s].double()
        q = t.sigmoid(u)
        dp = dout[s].double() * q * (1 + u * (1 - q))
        dw += t.matmul(dp.t().contiguous(), x[s].double())
        db += dp.sum(0)
    near("dbias", got["dbias"], db, "f32")
    d = got["dweight"].double() - dw
    assert float(d.norm() / dw.norm()) <= 4e-3

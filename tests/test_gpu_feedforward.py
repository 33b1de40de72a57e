"""GPU: the feed-forward layer's operators as they are used together: a layer
(norm with the residual stream, gated pair, projection back) and its gradients
against automatic differentiation in float64; its 8-bit prompt form and its
single-token form with 4-bit weights against the same layer on the weights that
the codes stand for; all of it captured and replayed; two streams at once."""
import pytest

import selective_state_space_mamba_amd as ms

from ffutil import close, maker, rows8, weights4
from scanutil import torch

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield
    torch().cuda.empty_cache()


def layer64(x, res, w, wg, wu, wd):
    """stream + down(silu(gate)·up), all float64; res may be None."""
    t = torch()
    s = x if res is None else x + res
    n = s / t.sqrt((s * s).mean(-1, keepdim=True) + EPS) * w
    g = n @ wg.t()
    h = g * t.sigmoid(g) * (n @ wu.t())
    return s + h @ wd.t()


def forward(v, **kw):
    n, stream, rstd = ms.rms_norm_fwd(v["x"], v["w"], v["res"], eps=EPS, **kw)
    h, pre = ms.gated_linear_fwd(n, v["wg"], v["wu"], want_pre=True, **kw)
    out, _ = ms.linear_fwd(h, v["wd"], None, stream, **kw)
    return out, (n, stream, rstd, h, pre)


def backward(v, kept, dout, **kw):
    n, stream, rstd, h, pre = kept
    gd = ms.linear_bwd(h, v["wd"], dout=dout, want_dbias=False, **kw)
    gg = ms.gated_linear_bwd(n, v["wg"], v["wu"], dout=gd["dx"], pre=pre, want_dbias=False, **kw)
    gn = ms.rms_norm_bwd(stream, v["w"], dout=gg["dx"], rstd=rstd, dadded=dout, **kw)
    return dict(x=gn["dx"], res=gn["dresidual"], w=gn["dweight"], wg=gg["dw_gate"], wu=gg["dw_up"], wd=gd["dweight"])


def make(M, D, H, dtype, seed):
    n = maker(seed)
    return dict(x=n((M, D), dtype), res=n((M, D), dtype), w=1 + n((D,), std=0.2), wg=n((H, D), dtype, D ** -0.5),
                wu=n((H, D), dtype, D ** -0.5), wd=n((D, H), dtype, H ** -0.5)), n((M, D), dtype)


@pytest.mark.parametrize("case", [(5, 64, 136, "f32"), (5, 64, 136, "bf16"), (700, 200, 520, "f32"), (700, 200, 520, "bf16"),
                                  (3000, 768, 2048, "bf16")], ids=lambda c: "%dx%dx%d-%s" % c)
def test_training_layer(case):
    """bfloat16: the layer rounds the stream, n, h, dh, dn and what enters the products, each by 1.1e-3 in L2 of what
    it is; a gradient passes at most six of them and its own, sqrt(7)·1.1e-3 = 3e-3 where nothing cancels: 1e-2."""
    M, D, H, dtype = case
    print("[gpu case] layer", case, flush=True)
    v, dout = make(M, D, H, dtype, M)
    out, kept = forward(v)
    g = backward(v, kept, dout)
    ref = {k: a.double().requires_grad_(True) for k, a in v.items()}
    want = layer64(**ref)
    want.backward(dout.double())
    for name, got, exact in [("out", out, want.detach())] + [(k, g[k], ref[k].grad) for k in v]:
        d = got.double() - exact
        rel = float(d.norm() / exact.norm())
        print("%s: %.2e" % (name, rel), flush=True)
        assert rel <= (1e-2 if dtype == "bf16" else 2e-5), (name, rel)


@pytest.mark.parametrize("M", [1, 9, 300])
def test_8bit_prompt_form(M):
    """The norm's 8-bit rows and 8-bit weights: against the same rows and weights in float64, to the output's rounding;
    against the layer without quantised rows, within the rows' step (2^-4/sqrt(3) = 3.6e-2 of the product in L2)."""
    t = torch()
    v, _ = make(M, 256, 512, "bf16", M)
    w8, sw = rows8(v["wg"].float())
    q, scale, stream = ms.rms_norm_q8(v["x"], v["w"], v["res"], eps=EPS)
    got = ms.linear_q8(q, scale, w8, sw, act=ms.ACT_SILU)
    u = t.matmul(q.double() * scale.double()[:, None], (w8.double() * sw.double()[:, None]).t().contiguous())
    close("products", got, u * t.sigmoid(u), "bf16")
    n, added, _ = ms.rms_norm_fwd(v["x"], v["w"], v["res"], eps=EPS)
    assert t.equal(added, stream)
    full, _ = ms.linear_fwd(n, (w8.float() * sw[:, None]).bfloat16())
    plain = ms.linear_q8(q, scale, w8, sw)
    rel = float((plain.double() - full.double()).norm() / full.double().norm())
    print("against the unquantised rows: %.2e" % rel, flush=True)
    assert rel <= 3.6e-2 + 1e-2


@pytest.mark.parametrize("M", [1, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_single_token_form(M, dtype):
    """norm -> 4-bit projection -> 4-bit projection back onto the stream, against float64 on what the codes stand for."""
    t = torch()
    D, H = 256, 544
    v, _ = make(M, D, H, dtype, M)
    up, down = weights4(H, D, 64, 1, True), weights4(D, H, 128, 2, False)
    n, stream, _ = ms.rms_norm_fwd(v["x"], v["w"], v["res"], eps=EPS)
    h = ms.linear_q4(n, *up[:3], group=64, act=ms.ACT_GELU)
    out = ms.linear_q4(h, *down[:3], None, stream, group=128)
    s = v["x"].double() + v["res"].double()
    nn = s / t.sqrt((s * s).mean(-1, keepdim=True) + EPS) * v["w"].double()
    u = nn @ up[3].t()
    want = s + (0.5 * u * t.special.erfc(-u / 2 ** 0.5)) @ down[3].t()
    close("out", out, want, "f32" if dtype == "f32" else "bf16 grad")  # (the stream's rounding and its own)


def test_captured_together_with_shared_weights():
    """A training step and a single-token step captured in two graphs, replayed in turn with new inputs."""
    t = torch()
    v, dout = make(300, 128, 264, "bf16", 3)
    tok, _ = make(4, 128, 264, "bf16", 4)
    q4 = weights4(128, 128, 32, 5, True)[:3]

    def step():
        out, kept = forward(v)
        return [out] + list(backward(v, kept, dout).values())

    def token():
        n, stream, _ = ms.rms_norm_fwd(tok["x"], v["w"], tok["res"], eps=EPS)
        h, _ = ms.gated_linear_fwd(n, v["wg"], v["wu"])
        out, _ = ms.linear_fwd(h, v["wd"], None, stream)
        q, scale, _ = ms.rms_norm_q8(out, v["w"], eps=EPS)
        return [out, scale, ms.linear_q4(out, *q4, group=32)]

    step(), token()
    t.cuda.synchronize()
    ga, gb = t.cuda.CUDAGraph(), t.cuda.CUDAGraph()
    with t.cuda.graph(ga):
        a = step()
    with t.cuda.graph(gb):
        b = token()
    n = maker(6)
    for k in range(3):
        v["x"].copy_(n((300, 128), "bf16"))
        tok["x"].copy_(n((4, 128), "bf16"))
        ga.replay()
        gb.replay()
        t.cuda.synchronize()
        assert float(t.randn(1 << 20, device="cuda:0").sum()) == pytest.approx(0, abs=1e5)
        assert all(t.equal(p, q) for p, q in zip(a, step())), k
        assert all(t.equal(p, q) for p, q in zip(b, token())), k


def test_two_streams_at_once():
    t = torch()
    v, dout = make(1500, 256, 520, "bf16", 7)
    u, eout = make(1100, 256, 520, "bf16", 8)
    want = []
    for a, d in ((v, dout), (u, eout)):
        out, kept = forward(a)
        want.append([out] + list(backward(a, kept, d).values()))
    t.cuda.synchronize()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, (a, d) in zip(streams, ((v, dout), (u, eout))):
            out, kept = forward(a, stream=s)
            got.append([out] + list(backward(a, kept, d, stream=s).values()))
        t.cuda.synchronize()
        assert all(t.equal(p, q) for g, w in zip(got, want) for p, q in zip(g, w))



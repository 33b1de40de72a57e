"""GPU parity of the root-mean-square norm with the residual's addition
(mamba_rms_norm_*) with its float64 form, element by element.

Tolerances, written before the first run.  The mean of D squares, in float32 in
chains of at most 4 vectors of 8 and 10 joins of positive terms, is off by at
most 50·2^-24 relative, rstd by half of it and two roundings more, xh and y by
three more: 2^-19 covers each.  A bfloat16 output adds half a step, 2^-8, an
8-bit one 2^-4 (2^-10 absolute below 2^-6, where the steps are 2^-9).  mean(t·xh)
errs by the same chains relative to the mean of |t·xh|, and each term of ds by a
few roundings: 2^-18 of the terms' magnitudes.  dweight is a sum over rows in
chains of at most rows/512 + 4 + 32 + 16 terms, each with xh's error: 2^-17 of
its terms' magnitudes for up to 70000 rows."""
import pytest

import selective_state_space_mamba_amd as ms

from ffutil import HALF, dtype_of, maker, rms_grads, rms_ref, within
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


def check_fwd(x, w, res, got, dtype, eps=EPS):
    out, added, rstd = got
    s, r, y = rms_ref(x, w, res, eps)
    if res is None:
        assert added is None
    else:
        assert torch().equal(added, s)
    within("rstd", rstd, r, r * 2.0 ** -19)
    within("out", out, y, y.abs() * (HALF[dtype] + 2.0 ** -19))
    return s, r, y


def check_q8(y, got):
    t = torch()
    q, scale, _ = got
    assert q.dtype is t.float8_e4m3fn
    want = (y.abs().amax(-1) / 448).clamp(min=2.0 ** -100)
    within("scale", scale, want, want * 2.0 ** -19)
    v = y / want[..., None]
    within("q", q.float(), v, t.maximum(v.abs() * HALF["e4m3"], t.full_like(v, 2.0 ** -10)) + v.abs() * 2.0 ** -18)


CASES = [(M, D, ty, rt) for (M, D), types in {
    (1, 1): 3, (3, 7): 3, (5, 8): 3, (2, 40): 1, (300, 63): 3, (257, 512): 1, (9, 513): 2, (64, 1000): 3, (700, 1536): 1,
    (5, 1536): 3, (256, 520): 1, (257, 520): 1, (1000, 2048): 3, (1000, 2049): 3, (33, 4096): 1, (70, 5001): 3,
    (40, 6144): 2, (21, 8192): 3, (11, 8200): 3, (4, 16383): 3, (6, 16384): 3, (5003, 768): 3, (4097, 24): 1,
    (3000, 1029): 2, (300, 777): 3, (1100, 1999): 2, (30, 7001): 2, (1025, 1280): 1, (130, 640): 2, (1024, 776): 3, (1025, 776): 3, (512, 129): 1, (1024, 40): 1,
    (70001, 64): 1, (9001, 128): 3, (5003, 106): 3, (2001, 250): 3, (1203, 256): 3, (613, 9): 2}.items()
    for ty, rt in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"))[:types]]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%d-%s-%s" % c)
def test_forward_8bit_and_gradients(case):
    M, D, dtype, rtype = case
    print("[gpu case] rms", case, flush=True)
    t = torch()
    n = maker(M * 31 + D)
    x, res, w = n((M, D), dtype), n((M, D), rtype, 3.0), 1 + n((D,), std=0.2)
    dout, dadded = n((M, D), dtype), n((M, D), rtype)
    for wt, rs in ((w, res), (None, res), (w, None)):
        got = ms.rms_norm_fwd(x, wt, rs, eps=EPS)
        s, r, y = check_fwd(x, wt, rs, got, dtype)
        q = ms.rms_norm_q8(x, wt, rs, eps=EPS)
        check_q8(y, q)
        assert rs is None or t.equal(q[2], s)
        rstd = got[2]
        for da in ((dadded, None) if rs is not None else (None,)):
            g = ms.rms_norm_bwd(s, wt, dout=dout, rstd=rstd, dadded=da)
            ds, size, dw, dwsize = rms_grads(s, wt, r, dout, da)
            within("dx", g["dx"], ds, size * 2.0 ** -18 + ds.abs() * HALF[dtype])
            assert g["dx"].dtype is dout.dtype and g["dresidual"].dtype is s.dtype
            if s.dtype is dout.dtype:
                assert g["dresidual"] is g["dx"]
            else:
                within("dresidual", g["dresidual"], ds, size * 2.0 ** -18)
            if wt is None:
                assert g["dweight"] is None
            else:
                within("dweight", g["dweight"], dw, dwsize * 2.0 ** -17 + 1e-300)
            again = ms.rms_norm_bwd(s, wt, dout=dout, rstd=rstd, dadded=da)
            assert all(a is None or t.equal(a, g[k]) for k, a in again.items())
            alone = ms.rms_norm_bwd(s, wt, dout=dout, rstd=rstd, dadded=da, want_dweight=False)
            assert alone["dweight"] is None and t.equal(alone["dx"], g["dx"])


@pytest.mark.parametrize("D", [48, 1001, 4096])
def test_in_place_leading_axes_and_slices(D):
    t = torch()
    n = maker(D)
    x, res, w = n((2, 3, D), "bf16"), n((2, 3, D), "bf16"), n((D,))
    out, added, rstd = ms.rms_norm_fwd(x, w, res)
    assert out.shape == x.shape and rstd.shape == (2, 3)
    x2, r2 = x.clone(), res.clone()
    o2, a2, s2 = ms.rms_norm_fwd(x2, w, r2, out=x2, added=r2)
    assert o2 is x2 and a2 is r2 and t.equal(o2, out) and t.equal(a2, added) and t.equal(s2, rstd)
    # tensors that begin off 16 bytes, by each element
    for off in range(1, 9):
        def moved(v):
            buf = t.zeros(v.numel() + off, dtype=v.dtype, device=v.device)
            buf[off:] = v.reshape(-1)
            return buf[off:].view(v.shape)
        o3, a3, s3 = ms.rms_norm_fwd(moved(x), moved(w), moved(res))
        # (the same sums in the same order: the rows' vectors are the same)
        assert t.equal(o3, out) and t.equal(a3, added) and t.equal(s3, rstd)
        q = ms.rms_norm_q8(x, w, res)
        q3 = ms.rms_norm_q8(moved(x), moved(w), moved(res), out=moved(q[0].view(t.uint8)).view(t.float8_e4m3fn))
        assert t.equal(q3[0].view(t.uint8), q[0].view(t.uint8)) and t.equal(q3[1], q[1])
        dout = n((2, 3, D), "bf16")
        g = ms.rms_norm_bwd(added, w, dout=dout, rstd=rstd, dadded=x)
        g3 = ms.rms_norm_bwd(moved(added), moved(w), dout=moved(dout), rstd=rstd, dadded=moved(x))
        assert t.equal(g3["dx"], g["dx"]) and t.equal(g3["dweight"], g["dweight"])


def test_nothing_beside_the_rows_is_written():
    """A guard on either side of every output, at sizes that end inside a vector."""
    t = torch()
    for M, D in ((3, 5), (7, 1003), (2, 16381)):
        n = maker(D)
        x, res, w = n((M, D), "bf16"), n((M, D)), n((D,))

        def guarded(dtype, shape):
            size = 1
            for v in shape:
                size *= v
            buf = t.full((size + 128,), 77, dtype=t.uint8, device="cuda:0").to(dtype) if dtype != t.float8_e4m3fn \
                else t.full((size + 128,), 77, dtype=t.uint8, device="cuda:0")
            mid = buf[64:64 + size]
            return buf, (mid.view(t.float8_e4m3fn) if dtype == t.float8_e4m3fn else mid).view(shape)

        bufs = {}
        for name, dt, shape in (("out", t.bfloat16, (M, D)), ("added", t.float32, (M, D)), ("rstd", t.float32, (M,))):
            bufs[name] = guarded(dt, shape)
        ms.rms_norm_fwd(x, w, res, **{k: v[1] for k, v in bufs.items()})
        bufs8 = {"out": guarded(t.float8_e4m3fn, (M, D)), "scale": guarded(t.float32, (M,))}
        ms.rms_norm_q8(x, w, res, **{k: v[1] for k, v in bufs8.items()})
        for b in (bufs, bufs8):
            for name, (buf, _) in b.items():
                assert bool((buf[:64].float() == 77).all()) and bool((buf[-64:].float() == 77).all()), (M, D, name)


@pytest.mark.parametrize("D", [96, 1001, 2056])
def test_zeros_nan_and_infinity_stay_in_their_rows(D):
    t = torch()
    n = maker(D)
    x, w = n((40, D), "bf16"), 1 + n((D,), std=0.2)
    want = ms.rms_norm_fwd(x, w)
    wq = ms.rms_norm_q8(x, w)
    x[3] = 0
    x[7, D - 1] = float("nan")
    x[39, 0] = float("inf")
    out, _, rstd = ms.rms_norm_fwd(x, w)
    q, scale, _ = ms.rms_norm_q8(x, w)
    good = [m for m in range(40) if m not in (3, 7, 39)]
    assert t.equal(out[good], want[0][good]) and t.equal(scale[good], wq[1][good])
    assert t.equal(q.view(t.uint8)[good], wq[0].view(t.uint8)[good])
    assert bool((out[3] == 0).all()) and abs(float(rstd[3]) - EPS ** -0.5) <= 1e-5 * EPS ** -0.5
    assert bool((q[3].float() == 0).all()) and float(scale[3]) == 2.0 ** -100
    assert bool(out[7].isnan().all()) and bool(q[7].float().isnan().all()) and bool(scale[7].isnan())
    # an infinity: rstd is 0, its own place 0·inf, the others 0
    assert bool(out[39, 0].isnan()) and bool((out[39, 1:] == 0).all()) and float(rstd[39]) == 0
    assert bool(q[39].float().isnan().all())
    # gradients of a row with a NaN: that row's, and dweight's
    dout = n((40, D), "bf16")
    g = ms.rms_norm_bwd(x, w, dout=dout, rstd=rstd)
    assert bool(g["dx"][7].isnan().all()) and bool(g["dx"][good].isfinite().all())


def test_tiny_and_large_values():
    """Rows of 2^-60 (eps decides), and 8-bit rows whose scale would vanish."""
    t = torch()
    x = t.full((2, 64), 2.0 ** -60, device="cuda:0")
    out, _, rstd = ms.rms_norm_fwd(x, eps=1e-5)
    within("rstd", rstd, t.full((2,), 1e-5 ** -0.5, device="cuda:0").double(), t.full((2,), 1e-3, device="cuda:0").double())
    _, rstd, y = rms_ref(x, None, None, 0.0)  # 2^-120 is a normal float32
    out, _, r0 = ms.rms_norm_fwd(x, eps=0.0)
    within("out", out, y, y * 2.0 ** -19)
    w = t.full((64,), 1e-38, device="cuda:0")
    q, scale, _ = ms.rms_norm_q8(x, w, eps=0.0)
    assert bool((scale == 2.0 ** -100).all())
    v = 1e-38 * 2.0 ** 100  # 1.3e-8: below half the smallest 8-bit step
    assert v < 2.0 ** -10 and bool((q.float() == 0).all())
    big = t.full((1, 64), 1e17, device="cuda:0")
    out, _, _ = ms.rms_norm_fwd(big)
    within("big", out, t.ones(1, 64, device="cuda:0").double(), t.full((1, 64), 2.0 ** -19, device="cuda:0").double())


def test_gradients_against_differences():
    """Central differences of the kernel's float32 forward along the gradient's signs: rounding over the step leaves
    about 1e-3 of the derivative, 1e-2 is asked."""
    t = torch()
    for D in (24, 1001):
        n = maker(D)
        x, res, w = n((7, D)), n((7, D)), 1 + n((D,), std=0.2)
        dout, dadded = n((7, D)), n((7, D))

        def loss(x, res, w):
            out, added, _ = ms.rms_norm_fwd(x, w, res)
            return float((out.double() * dout.double()).sum() + (added.double() * dadded.double()).sum())

        _, added, rstd = ms.rms_norm_fwd(x, w, res)
        g = ms.rms_norm_bwd(added, w, dout=dout, rstd=rstd, dadded=dadded)
        v = dict(x=x, res=res, w=w)
        for k, gk in (("x", "dx"), ("res", "dresidual"), ("w", "dweight")):
            d = t.sign(g[gk])
            eps = 2e-3
            num = (loss(**dict(v, **{k: v[k] + eps * d})) - loss(**dict(v, **{k: v[k] - eps * d}))) / (2 * eps)
            want = float((g[gk].double() * d.double()).sum())
            assert abs(num - want) <= 1e-2 * abs(want), (D, k, num, want)


def test_other_stream_and_graph():
    t = torch()
    for M, D in ((6, 1536), (5000, 264)):
        n = maker(M)
        x, res, w, dout = n((M, D), "bf16"), n((M, D)), n((D,)), n((M, D), "bf16")

        def both(**kw):
            out, added, rstd = ms.rms_norm_fwd(x, w, res, **kw)
            q, scale, _ = ms.rms_norm_q8(x, w, res, **kw)
            g = ms.rms_norm_bwd(added, w, dout=dout, rstd=rstd, **kw)
            return [out, added, rstd, q.view(t.uint8), scale, g["dx"], g["dresidual"], g["dweight"]]

        want = both()
        t.cuda.synchronize()
        s = t.cuda.Stream()
        got = both(stream=s)
        s.synchronize()
        assert all(t.equal(a, b) for a, b in zip(got, want))
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            got = both()
        for k in range(3):
            for v in got:
                v.zero_()
            x.copy_(n((M, D), "bf16"))
            graph.replay()
            t.cuda.synchronize()
            junk = t.randn(1 << 20, device="cuda:0").sum().item()
            assert junk == junk
            assert all(t.equal(a, b) for a, b in zip(got, both())), k


def test_more_elements_than_32_bits_count():
    t = torch()
    D = 2048
    M = (1 << 31) // D + 37
    print("[gpu case] rms rows", M, D, flush=True)
    n = maker(1)
    part = n((64, D), "bf16")
    x = t.empty(M, D, dtype=t.bfloat16, device="cuda:0")
    x.view(-1, D)[: M // 64 * 64].view(-1, 64, D)[:] = part
    x[M // 64 * 64:] = part[: M % 64]
    w = n((D,))
    out, _, rstd = ms.rms_norm_fwd(x, w)
    # (1088 rows of it: up to 1024 are summed up by more waves each, in another order)
    some = x[:1088].clone()
    want, _, wr = ms.rms_norm_fwd(some, w)
    assert t.equal(out[M // 64 * 64:], want[: M % 64]) and t.equal(rstd[-(M % 64):], wr[: M % 64])
    assert t.equal(out[:1088], want)
    q, scale, _ = ms.rms_norm_q8(x, w)
    wq = ms.rms_norm_q8(some, w)
    assert t.equal(q[M // 64 * 64:].view(t.uint8), wq[0][: M % 64].view(t.uint8)) and t.equal(scale[:1088], wq[1])
    g = ms.rms_norm_bwd(x, w, dout=x, rstd=rstd)
    wg = ms.rms_norm_bwd(some, w, dout=some, rstd=wr)
    assert t.equal(g["dx"][M // 64 * 64:], wg["dx"][: M % 64])


def test_more_rows_than_an_axis_of_workgroups():
    t = torch()
    M = (1 << 24) * 4 + 9  # four rows a workgroup of 256 threads: 2^32 threads and more
    x = t.ones(M, 1, dtype=t.bfloat16, device="cuda:0")
    x[-1] = -3
    out, _, rstd = ms.rms_norm_fwd(x, eps=0.0)
    assert float(out[-1]) == -1 and bool((out[:-1] == 1).all()) and abs(float(rstd[-1]) - 1 / 3) < 1e-6
    g = ms.rms_norm_bwd(x, t.ones(1, device="cuda:0"), dout=x, rstd=rstd)
    assert bool((g["dx"].float().abs() <= 2.0 ** -20).all())


def test_binding_refusals():
    t = torch()
    z = lambda *s, dtype=t.float32: t.zeros(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    x = z(4, 64)
    with pytest.raises(TypeError):
        ms.rms_norm_fwd(x.half())
    with pytest.raises(TypeError):  # a stream narrower than x
        ms.rms_norm_fwd(x, None, x.bfloat16())
    with pytest.raises(ValueError):
        ms.rms_norm_fwd(x, z(63))
    with pytest.raises(TypeError):
        ms.rms_norm_fwd(x.bfloat16(), z(64, dtype=t.bfloat16))
    with pytest.raises(ValueError):
        ms.rms_norm_fwd(z(64, 4).t())
    with pytest.raises(ValueError):
        ms.rms_norm_fwd(x, residual=z(4, 63))
    with pytest.raises(ValueError):
        ms.rms_norm_fwd(x, added=z(4, 64))
    with pytest.raises(TypeError):
        ms.rms_norm_fwd(x, residual=x, added=x.bfloat16())
    with pytest.raises(TypeError):
        ms.rms_norm_q8(x, out=z(4, 64))
    with pytest.raises(ms.MambaError):
        ms.rms_norm_fwd(x[:0])
    with pytest.raises(ms.MambaError):
        ms.rms_norm_fwd(x, eps=-1.0)
    with pytest.raises(ms.MambaError):
        ms.rms_norm_fwd(z(1, 16385))
    with pytest.raises(ValueError):
        ms.rms_norm_bwd(x, dout=z(4, 63), rstd=z(4))
    with pytest.raises(ValueError):
        ms.rms_norm_bwd(x, dout=x, rstd=z(5))
    with pytest.raises(TypeError):
        ms.rms_norm_bwd(x, dout=x.bfloat16(), rstd=z(4), dadded=x.bfloat16())
    with pytest.raises(ValueError):
        ms.rms_norm_fwd(t.zeros(4, 64))

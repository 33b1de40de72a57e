"""GPU: what the gated recurrence does where decays vanish, where a value is NaN
and where a sequence spans several blocks of tiles, with the float64 form."""
import numpy as np
import pytest

import selective_state_space_mamba_amd as ms

from layerutil import from_dev, glr_grads, glr_ref, to_dev
from scanutil import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch().cuda.is_available():
        pytest.skip("no GPU")
    ms.load_library()
    yield


def bits(t_):
    """NaNs compare equal."""
    t = torch()
    return t.nan_to_num(t_.float(), nan=12345.0, posinf=1e38, neginf=-1e38)


@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("with_lam", [False, True])
@pytest.mark.parametrize("shape", [(1, 700, 64), (3, 1500, 40), (40, 200, 1664)], ids=lambda s: "%dx%dx%d" % s)
def test_a_vanishing_decay_is_no_reset(shape, with_lam, reverse):
    """Decays of 0, and products of decays that underflow, still pass a NaN on: 0·NaN.  Only a reset stops one, and
    with a mask that holds none the results are those without a mask."""
    B, L, D = shape
    print("[gpu case] glr vanishing decays", shape, with_lam, reverse, flush=True)
    r = np.random.Generator(np.random.PCG64([L, D]))
    v = {k: r.standard_normal((B, L, D)).astype(np.float32) for k in "xiz"}
    v["r"] = r.choice(np.float32([30.0, 2.0, -1.0] if with_lam else [-200.0, -20.0, -3.0]), (B, L, D))
    lam = np.full(D, 30.0, np.float32) if with_lam else None
    dout = r.standard_normal((B, L, D)).astype(np.float32)
    bad = L // 7 if not reverse else L - 1 - L // 7  # a quarter into the scan, and near its end for the adjoint
    far = L - 1 - bad
    v["x"][:, bad, ::2] = np.nan
    dout[:, far, ::3] = np.nan
    a = [to_dev(v[k]) for k in "xriz"] + [to_dev(lam)]
    kw = dict(reverse=reverse)
    plain = ms.glr_fwd(*a, **kw)
    grads = ms.glr_bwd(*a, dout=to_dev(dout), **kw)
    none = to_dev(np.zeros((B, L), np.uint8))
    masked = ms.glr_fwd(*a, reset=none, **kw)
    mgrads = ms.glr_bwd(*a, dout=to_dev(dout), reset=none, **kw)
    for x, y in zip(plain, masked):
        assert torch().equal(bits(x), bits(y))
    for k in grads:
        assert grads[k] is None or torch().equal(bits(grads[k]), bits(mgrads[k])), k
    for reset in (None, np.zeros((B, L), np.uint8)):
        if reset is not None:
            reset[:, L // 2] = 1
        rd = None if reset is None else to_dev(reset)
        out, last = ms.glr_fwd(*a, reset=rd, **kw)
        g = ms.glr_bwd(*a, dout=to_dev(dout), reset=rd, **kw)
        with np.errstate(all="ignore"):
            ref = [v[k].astype(np.float64) for k in "xriz"] + [None if lam is None else lam.astype(np.float64)]
            want, want_last, _, _ = glr_ref(*ref, reverse=reverse, reset=reset)
            wg = glr_grads(*ref, dout.astype(np.float64), reverse=reverse, reset=reset)
        assert np.array_equal(np.isnan(from_dev(out)), np.isnan(want))
        assert np.array_equal(np.isnan(from_dev(last)), np.isnan(want_last))
        for k, w in wg.items():
            if w is not None:
                assert np.array_equal(np.isnan(from_dev(g[k])), np.isnan(w)), k


@pytest.mark.parametrize("rule", [ms.GLR_SQRT, ms.GLR_LERP, ms.GLR_UNIT])
def test_nan_in_lam_shows_in_its_channel(rule):
    """And in no other.  (The unit rule's first state does not depend on lam.)"""
    t = torch()
    B, L, D = 2, 300, 72
    g = t.Generator(device="cuda:0")
    g.manual_seed(3)
    x, r, z, dout = (t.randn(B, L, D, generator=g, device="cuda:0") for _ in range(4))
    lam = t.full((D,), -4.0, device="cuda:0")
    bad = lam.clone()
    bad[[5, 70]] = float("nan")
    keep = [d for d in range(D) if d not in (5, 70)]
    init = t.randn(B, D, generator=g, device="cuda:0")
    print("[gpu case] glr NaN in lam", rule, flush=True)
    want = ms.glr_fwd(x, r, None, z, lam, input_rule=rule, initial_state=init)
    got = ms.glr_fwd(x, r, None, z, bad, input_rule=rule, initial_state=init)
    wg = ms.glr_bwd(x, r, None, z, lam, dout=dout, input_rule=rule, initial_state=init)
    gg = ms.glr_bwd(x, r, None, z, bad, dout=dout, input_rule=rule, initial_state=init)
    ws, gs = init.clone(), init.clone()
    wo = ms.glr_step(ws, x[:, 0].contiguous(), r[:, 0].contiguous(), None, z[:, 0].contiguous(), lam, input_rule=rule)
    go = ms.glr_step(gs, x[:, 0].contiguous(), r[:, 0].contiguous(), None, z[:, 0].contiguous(), bad, input_rule=rule)
    pairs = [(want[0], got[0]), (want[1], got[1]), (ws, gs), (wo, go)]
    pairs += [(wg[k], gg[k]) for k in ("dr", "dz", "dlam", "dinit")]
    for w, v in pairs:
        assert t.equal(v[..., keep], w[..., keep])
        assert bool(t.isnan(v[..., [5, 70]]).all())
    # dx needs the later adjoints alone: NaN but at the last token
    assert t.equal(gg["dx"][..., keep], wg["dx"][..., keep])
    assert bool(t.isnan(gg["dx"][:, :-1][..., [5, 70]]).all())


def test_softplus_keeps_its_relative_accuracy():
    """One token behind a fully open gate (r = 30: sigmoid rounds to 1) with x = 1 and a small scale shows the rate:
    out = 1 - exp(-scale·softplus(lam)) = scale·softplus(lam) to its second order.  An exponential and a reciprocal of
    one ulp each, a quotient's series and the products around them are about ten roundings of 2^-24: 6e-7, from
    lam = -80 (softplus = 2e-35) to 80, where a sum 1 + e or a rounded exponent would lose up to all of them."""
    t = torch()
    D, scale = 8192, 2.0 ** -10
    lam = np.linspace(-80.0, 80.0, D).astype(np.float32)
    lam[: D // 2] = np.linspace(-6.0, 2.0, D // 2).astype(np.float32)  # densely where the terms are of one size
    x, r = t.ones(1, 1, D, device="cuda:0"), t.full((1, 1, D), 30.0, device="cuda:0")
    print("[gpu case] glr softplus", flush=True)
    want = -np.expm1(-scale * np.logaddexp(0.0, lam.astype(np.float64)))
    big = want > 1e-30  # (below, float32 holds fewer bits)
    step = ms.glr_step(t.zeros(1, D, device="cuda:0"), x[0], r[0], lam=to_dev(lam), scale=scale, input_rule=ms.GLR_LERP)
    out, _ = ms.glr_fwd(x, r, lam=to_dev(lam), scale=scale, input_rule=ms.GLR_LERP)
    for got in (from_dev(out)[0, 0], from_dev(step)[0]):
        rel = np.abs(got - want)[big] / want[big]
        print("worst %.2e at lam %.2f" % (rel.max(), lam[big][rel.argmax()]), flush=True)
        assert rel.max() <= 6e-7


def test_scalars_are_read_on_every_call():
    """A scale or a rule given as a tensor counts with the value it has at the call."""
    t = torch()
    g = t.Generator(device="cuda:0")
    g.manual_seed(4)
    x, r = (t.randn(2, 64, generator=g, device="cuda:0") for _ in range(2))
    lam = t.zeros(64, device="cuda:0")
    scale, rule, act = t.tensor(8.0), t.tensor(ms.GLR_SQRT), t.tensor(ms.ACT_NONE)
    for s, k in ((8.0, ms.GLR_SQRT), (2.0, ms.GLR_SQRT), (2.0, ms.GLR_UNIT)):
        scale.fill_(s), rule.fill_(k)
        want = ms.glr_step(t.ones(2, 64, device="cuda:0"), x, r, lam=lam, scale=s, input_rule=k)
        for sc in (scale, scale.numpy()):
            got = ms.glr_step(t.ones(2, 64, device="cuda:0"), x, r, lam=lam, scale=sc, input_rule=rule)
            assert t.equal(got, want), (s, k)
    w = t.randn(64, 64, generator=g, device="cuda:0")
    for a in (ms.ACT_NONE, ms.ACT_SILU):  # an activation's backward needs a larger workspace
        act.fill_(a)
        _, pre = ms.linear_fwd(x, w, act=act, want_pre=True)
        got = ms.linear_bwd(x, w, dout=r, pre=pre, act=act)
        want = ms.linear_bwd(x, w, dout=r, pre=pre, act=a)
        assert all(t.equal(got[n], want[n]) for n in got)


@pytest.mark.parametrize("reverse", [False, True])
def test_slices_of_a_batch(reverse):
    """bfloat16 items of an odd number of tokens and D = 8k + 4 channels begin 8 bytes apart from 16; every one of them
    is a contiguous tensor and gives what the item by itself gives."""
    t = torch()
    B, L, D = 3, 333, 76
    g = t.Generator(device="cuda:0")
    g.manual_seed(6)
    v = {k: t.randn(B, L, D, generator=g, device="cuda:0").bfloat16() for k in ("x", "r", "i", "z", "dout")}
    lam = t.full((D,), -3.0, device="cuda:0")
    init = t.randn(1, D, generator=g, device="cuda:0")
    print("[gpu case] glr slices", flush=True)
    for b in range(B):
        got = []
        for take in (lambda a: a, lambda a: a.clone()):
            s = {k: take(a[b:b + 1]) for k, a in v.items()}
            assert s["x"].is_contiguous()
            args = (s["x"], s["r"], s["i"], s["z"], lam)
            out = take(t.empty(B, L, D, dtype=t.bfloat16, device="cuda:0")[b:b + 1])
            _, last, saved = ms.glr_fwd_save(*args, initial_state=init, reverse=reverse, out=out)
            grads = ms.glr_bwd(*args, dout=s["dout"], saved=saved, initial_state=init, reverse=reverse)
            state = init.clone()
            step = ms.glr_step(state, *(take(v[k][b, 7:8]) for k in "xriz"), lam, out=take(v["dout"][b, 7:8].clone()))
            got.append([out, last, step, state] + [grads[k] for k in sorted(grads)])
        assert all(t.equal(p, q) for p, q in zip(*got))


# Sequences of several blocks of tiles, forward (128 positions a tile) and backward (64), for each length of a block:
# 16 tiles below 8 rows (a batch item's 64 channels are one), 8 below 12, 4 from there on.
BLOCKS = [
    # B, L, D, dtype, rule, reverse, options                                   rows
    (7, 2500, 12, "f32", "lerp", False, dict(reset=0.002)),                   # 7
    (8, 2177, 20, "bf16", "sqrt", False, {}),                                 # 8
    (1, 2309, 640, "f32", "sqrt", False, {}),                                 # 10
    (1, 2309, 640, "bf16", "lerp", True, dict(reset=0.002)),                  # 10
    (11, 1100, 64, "f32", "unit", True, dict(reset=0.004, lam=False)),        # 11
    (12, 700, 8, "f32", "sqrt", True, {}),                                    # 12
    (3, 1500, 392, "f32", "sqrt", False, dict(reset=0.003)),                  # 21
    (3, 1500, 392, "bf16", "unit", True, dict(lam=False)),                    # 21
    (1, 1025, 1300, "f32", "lerp", False, dict(z=False, reset=0.003)),        # 21
    (2, 640, 2048, "bf16", "sqrt", False, {}),                                # 64: exactly 5 forward tiles, 10 backward
]


@pytest.mark.parametrize("case", BLOCKS, ids=lambda c: "B%d-L%d-D%d-%s-%s-rev%d" % c[:6])
def test_chains_of_several_blocks(case):
    """The tolerances of test_gpu_glr, whose inputs and checks these are."""
    import test_gpu_glr as base
    B, L, D, dtype, rule, reverse, opt = case
    print("[gpu case] glr blocks", case, flush=True)
    dev, ref = base.make(B, L, D, dtype, L + D, **opt)
    kw, rkw = base.kwargs(dev, rule, reverse, False), base.kwargs(ref, rule, reverse, True)
    out, last, saved = ms.glr_fwd_save(*base.args(dev), **kw)
    g = ms.glr_bwd(*base.args(dev), dout=dev["dout"], dlast=dev["dlast"], saved=saved, **kw)
    torch().cuda.synchronize()
    want, want_last, _, _ = glr_ref(*base.args(ref), **rkw)
    wg = glr_grads(*base.args(ref), ref["dout"], ref["dlast"], **rkw)
    base.close("out", from_dev(out), want, dtype)
    base.close("last_state", from_dev(last), want_last, "f32")
    for k, w in wg.items():
        assert (g[k] is None) == (w is None), k
        if w is not None:
            base.close(k, from_dev(g[k]), w, "f32" if k in ("dlam", "dinit") else dtype)


def test_overlapping_calls_on_two_streams():
    """Each waits in its own memory: what two streams run at once, and on one workspace each, is what one runs alone."""
    t = torch()
    gen = t.Generator(device="cuda:0")
    gen.manual_seed(8)

    def case(L, D):
        v = [t.randn(1, L, D, generator=gen, device="cuda:0").bfloat16() for _ in range(5)]
        lam = t.full((D,), -4.0, device="cuda:0")
        w = (t.randn(D, D, generator=gen, device="cuda:0") / D ** 0.5).bfloat16()

        def call(stream, ws):
            k = dict(stream=stream)
            n, mean, rstd = ms.group_norm_fwd(v[0], 4, act=ms.ACT_SILU, workspace=ws[0], **k)
            p, pre = ms.linear_fwd(n, w, act=ms.ACT_SILU, want_pre=True, workspace=ws[1], **k)
            out, last, saved = ms.glr_fwd_save(p, *v[1:4], lam, workspace=ws[2], **k)
            g = ms.glr_bwd(p, *v[1:4], lam, dout=v[4], saved=saved, workspace=ws[2], **k)
            d = ms.linear_bwd(n, w, dout=g["dx"], pre=pre, act=ms.ACT_SILU, workspace=ws[1], **k)
            e = ms.group_norm_bwd(v[0], 4, dout=d["dx"], mean=mean, rstd=rstd, act=ms.ACT_SILU, workspace=ws[0], **k)
            return [out, last, g["dr"], g["dlam"], d["dweight"], d["dbias"], e["dx"]]
        return call

    calls = [case(20000, 192), case(9000, 640)]
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    none = (None, None, None)
    print("[gpu case] two streams", flush=True)
    want = [c(None, none) for c in calls]
    t.cuda.synchronize()
    spaces = [[t.empty(64 << 20, dtype=t.uint8, device="cuda:0") for _ in range(3)] for _ in calls]
    t.cuda.synchronize()
    for ws in ([none, none], spaces):
        got = [[], []]
        for _ in range(5):
            for k, c in enumerate(calls):
                got[k].append(c(streams[k], ws[k]))
        t.cuda.synchronize()
        for k in range(2):
            for run in got[k]:
                assert all(t.equal(a, b) for a, b in zip(run, want[k]))

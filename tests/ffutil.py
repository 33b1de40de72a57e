"""Plain float64 references of the feed-forward layer's operators, for the
tests, in torch on whatever device the inputs are."""
import math

from scanutil import torch

# half a step of a type, relative to the value
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24, "e4m3": 2.0 ** -4}


def dtype_of(name):
    return {"bf16": torch().bfloat16, "f32": torch().float32}[name]


def maker(seed, device="cuda:0"):
    """normal(shape, type, std): seeded values of a type."""
    t = torch()
    g = t.Generator(device="cpu")
    g.manual_seed(seed)
    return lambda shape, dtype="f32", std=1.0: (t.randn(*shape, generator=g) * std).to(dtype_of(dtype)).to(device)


def act64(u, act):
    """The activation and its derivative."""
    t = torch()
    if act == "relu":
        return u.clamp(min=0), (u > 0).to(u.dtype)
    if act == "silu":
        q = t.sigmoid(u)
        return u * q, q * (1 + u * (1 - q))
    if act == "gelu":
        cdf = t.special.erfc(-u / math.sqrt(2)) / 2
        return u * cdf, cdf + u * t.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    return u, t.ones_like(u)


def rms_ref(x, w, res, eps):
    """s (as stored), rstd and y, float64."""
    t = torch()
    s = x if res is None else (x.float() + res.float()).to(res.dtype)
    v = s.double()
    rstd = 1 / t.sqrt((v * v).mean(-1) + eps)
    y = v * rstd[..., None]
    return s, rstd, y if w is None else y * w.double()


def rms_grads(s, w, rstd, dout, dadded):
    """ds, dweight and, for each, the sum of its terms' magnitudes."""
    v, dy = s.double(), dout.double()
    xh = v * rstd[..., None]
    tt = dy if w is None else dy * w.double()
    c = (tt * xh).mean(-1, keepdim=True)
    ds = rstd[..., None] * (tt - xh * c)
    size = rstd[..., None] * (tt.abs() + xh.abs() * (tt * xh).abs().mean(-1, keepdim=True))
    if dadded is not None:
        ds = ds + dadded.double()
        size = size + dadded.double().abs()
    axes = tuple(range(s.dim() - 1))
    return ds, size, (dy * xh).sum(axes), (dy * xh).abs().sum(axes)


def within(name, got, want, tol):
    """|got - want| <= tol, element by element."""
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    worst = float((d / tol.clamp(min=1e-300)).max()) if d.numel() else 0.0
    print("%s: worst %.3f of the tolerance" % (name, worst), flush=True)
    assert not bool(bad.any()), (name, worst)


# Products.  A float32 sum of K products errs by about sqrt(K)·2^-24 of its scale,
# 4e-6 at K = 4096: 2e-4 of the largest value and 2e-5 in the L2 norm.  bfloat16
# outputs carry one rounding (2^-9/sqrt(3) = 1.1e-3 in L2): 1e-2 and 3e-3;
# gradients behind an activation one more, of what enters the products: 4e-3.
TOL = {"f32": (2e-4, 2e-5), "bf16": (1e-2, 3e-3), "bf16 grad": (2e-2, 4e-3)}


def close(name, got, want, kind):
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert bool(got.isfinite().all()), name
    d = got.double() - want
    top, norm = float(want.abs().max()), float(want.norm())
    a, b = float(d.abs().max()) / (top or 1.0), float(d.norm()) / (norm or 1.0)
    print("%s: max %.2e l2 %.2e" % (name, a, b), flush=True)
    assert a <= TOL[kind][0] and b <= TOL[kind][1], (name, a, b)


def mm(a, b):
    """a·bᵀ in float64."""
    return torch().matmul(a.double(), b.double().t().contiguous())


def gated_ref(x, wg, wu, bg, bu, act, dout=None):
    """out, g, u and, for dout, the gradients."""
    g, u = mm(x, wg), mm(x, wu)
    if bg is not None:
        g = g + bg.double()
    if bu is not None:
        u = u + bu.double()
    a, da = act64(g, act)
    if dout is None:
        return a * u, g, u
    dg, du = dout.double() * u * da, dout.double() * a
    t = lambda v: v.t().contiguous()  # noqa: E731
    return a * u, g, u, dict(dx=mm(dg, t(wg)) + mm(du, t(wu)), dw_gate=mm(t(dg), t(x)), dw_up=mm(t(du), t(x)),
                             db_gate=dg.sum(0), db_up=du.sum(0))


def finish_ref(u, b, act, res):
    u = act64(u if b is None else u + b.double(), act)[0]
    return u if res is None else u + res.double()


def rows8(v):
    """Rows in e4m3 with their scales."""
    t = torch()
    scale = (v.float().abs().amax(1) / 448).clamp(min=1e-30)
    return (v.float() / scale[:, None]).to(t.float8_e4m3fn), scale


def weights4(N, K, group, seed, zero, scale_type="bf16", device="cuda:0"):
    """Packed weights, scale, zero, and what they stand for in float64."""
    t = torch()
    g = t.Generator(device="cpu")
    g.manual_seed(seed)
    G = -(-K // group)
    q = t.randint(0, 16, (N, K), generator=g, dtype=t.uint8)
    scale = (0.05 + 0.2 * t.rand(N, G, generator=g)).to(dtype_of(scale_type)) * (K ** -0.5)
    scale = scale.to(dtype_of(scale_type))
    z = t.randint(0, 16, (N, G), generator=g, dtype=t.uint8) if zero else None
    at = t.arange(K) // group
    w = (q.double() - (8.0 if z is None else z.double()[:, at])) * scale.double()[:, at]
    packed = q[:, 0::2] | (q[:, 1::2] << 4)
    return packed.contiguous().to(device), scale.to(device), None if z is None else z.to(device), w.to(device)


def planned(M, N, K, more=False, wide=True):
    """(tile rows, tile columns, shares, us) of a product of bfloat16 rows, written from the rule beside the launch
    (csrc/linear_launch.h): the least expected time.  more: of the gated pair (its N columns twice, without the
    192 columns of wide) and of 8-bit operands (half their K)."""
    best = None
    for bm, bn, slots, fix, per in ((128, 128, 512, 5.8, 0.0158), (256, 192, 256, 10.0 if more else 7.8, 0.0217),
                                    (256, 256, 256) + ((12.0, 0.025) if more else (6.4, 0.0293))):
        if bn == 192 and not wide:
            continue
        tiles, stages = -(-M // bm) * -(-N // bn), -(-K // 64)
        most = max(min(slots // tiles if tiles < slots else 1, stages // 8), 1)
        s = 1
        while True:
            each = -(-stages // s)
            shares = -(-stages // each)
            rounds = -(-tiles * shares // slots)
            last = 0.6 if bm == 128 and (tiles * shares - 1) % slots < 256 else 1.0
            us = rounds * fix + (rounds - 1 + last) * per * each * 64
            if shares > 1:
                us += 4.0 + shares * M * N * 8 / 5.0e6
            if best is None or us < best[3]:
                best = (bm, bn, shares, us)
            if s >= most:
                break
            s = min(2 * s, most)
    return best


def planned_kind(op, M, K, N):
    """How the forward of a "gated" pair of bfloat16 rows, or a product of "q8" operands, is run (the same rules):
    ("rows", tiles), ("long", stages) or ("tile", rows, columns, shares)."""
    gated = op == "gated"
    cols, k = (2 * N, K) if gated else (N, K // 2)
    tile = planned(M, cols, k, True, not gated)
    kind, best = ("tile",) + tile[:3], 0.9 * tile[3]
    if M <= 256:
        rounds = {tiles: -(-(-(-M // (16 * tiles)) * -(-N // 16)) // 256) for tiles in (1, 2, 4)}
        time, tiles = min((t * (1.0 + 0.6 * (rounds[n] - 1)), n) for n, t in ((1, 1.0), (2, 1.25), (4, 1.8)))
        time *= 2.6 + 2.8e-3 * K if gated else 2.7 + 0.9e-3 * K
        if M <= 64 or time < 0.8 * tile[3]:
            kind, best = ("rows", tiles), time
    groups = -(-M // 64) * -(-cols // 64)
    if groups <= 2048 and k >= 256:
        stages = 8 if groups <= 256 and k > 1024 else 4
        us = 5.0 + 0.0039 * k if stages == 8 else 6.0 + 0.003 * k
        if groups > 256:
            us = 1.5 + (4.5 + 0.006 * k) * -(-groups // 512)
        if us < best:
            kind = ("long", stages)
    return kind

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

"""The operators around the scan, as they are measured: the gated linear
recurrence, group normalisation with an activation (channels last), and the
matrix product with bias, activation and residual.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU,
``run`` makes one pass: with ``own`` false in elementary torch operations in 32
bits (rounded once, at the end), with ``own`` true through this repository's
entry points.  ``exact`` is the definition in 64 bits.

  glr      fwd / train / step   x, r, i, z [B][L][D], lam [D]
  gnorm    fwd / train          x [B][L][D] in G groups
  linear   fwd / train          x [M][K], weight [N][K]
"""
import math

import torch

own = False

SCALE = 8.0  # of the recurrence's decay rate
EPS = 1e-5   # of the normalisation


def listed():
    return [
        # One layer of a small language model in training or prefill: batch 8, 2048 tokens, 1536 channels,
        # both gates and the output gate.
        dict(name="glr fwd layer", op="glr", do="fwd", B=8, L=2048, D=1536, dtype="bf16", rule="sqrt", lam=True,
             gate=True, z=True, reset=False, reverse=False),
        # A single document of 262144 tokens: few rows, all the parallelism is along time.
        dict(name="glr fwd long", op="glr", do="fwd", B=1, L=262144, D=2048, dtype="bf16", rule="sqrt", lam=True,
             gate=True, z=True, reset=False, reverse=False),
        # The layer's training step: forward, then every gradient.
        dict(name="glr train layer", op="glr", do="train", B=8, L=2048, D=1536, dtype="bf16", rule="sqrt", lam=True,
             gate=True, z=True, reset=False, reverse=False),
        # Packed documents of odd total length in float32, no output gate, the complementary input rule, scanned
        # from the end.
        dict(name="glr train packed f32", op="glr", do="train", B=3, L=4133, D=392, dtype="f32", rule="lerp",
             lam=False, gate=True, z=False, reset=True, reverse=True),
        # One token of each of 8 sequences: the decode step, where latency counts.
        dict(name="glr step", op="glr", do="step", B=8, L=1, D=1536, dtype="bf16", rule="sqrt", lam=True, gate=True,
             z=True, reset=False, reverse=False),
        # Normalisation before a cross scan: 64 x 64 maps of 192 channels, 6 channels a group, batch 32.
        dict(name="gnorm fwd map", op="gnorm", do="fwd", B=32, L=4096, D=192, G=32, dtype="bf16", act="silu"),
        # Normalisation of every token over heads of 64 channels: 8 x 2048 tokens.
        dict(name="gnorm fwd token", op="gnorm", do="fwd", B=16384, L=1, D=1536, G=24, dtype="bf16", act="none"),
        # The maps' training step.
        dict(name="gnorm train map", op="gnorm", do="train", B=32, L=4096, D=192, G=32, dtype="bf16", act="silu"),
        # Expansion from 768 to 1536 channels with SiLU for 8 x 2048 tokens.
        dict(name="linear fwd expand", op="linear", do="fwd", M=16384, K=768, N=1536, dtype="bf16", act="silu",
             bias=True, residual=False),
        # Projection back onto the residual stream for 65536 tokens of 2048 channels.
        dict(name="linear fwd residual", op="linear", do="fwd", M=65536, K=2048, N=2048, dtype="bf16", act="none",
             bias=True, residual=True),
        # The same projection of 1536 to 768 channels for the one new token of each of 8 sequences.
        dict(name="linear step", op="linear", do="fwd", M=8, K=1536, N=768, dtype="bf16", act="none", bias=True,
             residual=True),
        # The expansion's training step: forward, then the gradients of input, weight and bias.
        dict(name="linear train expand", op="linear", do="train", M=16384, K=768, N=1536, dtype="bf16", act="silu",
             bias=True, residual=False),
    ]


def _log_int(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n == 3072 else n


def _eights(rng, lo, hi):
    """A multiple of 8, spread over the logarithm."""
    n = 8 * _log_int(rng, lo // 8, hi // 8)
    return n + 8 if n == 3072 else n


def draw(rng):
    op = rng.choice(["glr", "glr", "gnorm", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "glr":
        do = rng.choice(["fwd", "train", "step"])
        D = _eights(rng, 8, 4096)
        B = _log_int(rng, 1, 64)
        L = 1 if do == "step" else _log_int(rng, 1, max(1, min(65536, (1 << 25) // (B * D))))
        return dict(op=op, do=do, B=B, L=L, D=D, dtype=dtype, rule=rng.choice(["sqrt", "lerp", "unit"]),
                    lam=rng.random() < 0.7, gate=rng.random() < 0.7, z=rng.random() < 0.7,
                    reset=do != "step" and rng.random() < 0.4, reverse=do != "step" and rng.random() < 0.3)
    if op == "gnorm":
        G = rng.choice([1, 2, 4, 8, 16, 24, 32])
        c = _log_int(rng, 1, max(1, 2048 // G))
        while (G * c) % 8 or G * c == 3072:
            c += 1
        D = G * c
        token = rng.random() < 0.4  # one token an item, or one map an item
        L = 1 if token else _log_int(rng, 2, max(2, min(16384, (1 << 24) // D)))
        B = _log_int(rng, 1, max(1, min(32768 if token else 64, (1 << 25) // (L * D))))
        return dict(op=op, do=rng.choice(["fwd", "train"]), B=B, L=L, D=D, G=G, dtype=dtype,
                    act=rng.choice(["none", "relu", "silu", "gelu"]))
    K, N = _eights(rng, 8, 4096), _eights(rng, 8, 4096)
    M = _log_int(rng, 1, max(1, min(16384, (1 << (34 if dtype == "bf16" else 32)) // (K * N))))
    return dict(op=op, do=rng.choice(["fwd", "train"]), M=M, K=K, N=N, dtype=dtype,
                act=rng.choice(["none", "relu", "silu", "gelu"]), bias=rng.random() < 0.7,
                residual=rng.random() < 0.5)


# ---- inputs ----

def prepare(case, seed):
    dev = "cuda:0"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s = dict(case=case)

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    if case["op"] == "glr":
        B, L, D = case["B"], case["L"], case["D"]
        shape = (B, D) if case["do"] == "step" else (B, L, D)
        s["x"], s["r"] = normal(*shape), normal(*shape)
        s["i"] = normal(*shape) if case["gate"] else None
        s["z"] = normal(*shape) if case["z"] else None
        # decay at a fully open gate between 0.9 and 0.999
        a = 0.9 + 0.099 * torch.rand(D, generator=g, device=dev)
        s["lam"] = torch.log(torch.expm1(-torch.log(a) / SCALE)) if case["lam"] else None
        s["init"] = normal(B, D, dtype=torch.float32)
        s["reset"] = None
        if case["reset"]:  # documents of about 200 tokens
            s["reset"] = (torch.rand(B, L, generator=g, device=dev) < 0.005).to(torch.uint8)
        if case["do"] == "train":
            s["dout"] = normal(*shape)
    elif case["op"] == "gnorm":
        B, L, D = case["B"], case["L"], case["D"]
        # activations with an offset of their own in every channel
        s["x"] = (normal(B, L, D, dtype=torch.float32) + normal(D, dtype=torch.float32)).to(dt)
        s["w"] = 1.0 + normal(D, dtype=torch.float32, std=0.2)
        s["b"] = normal(D, dtype=torch.float32, std=0.2)
        if case["do"] == "train":
            s["dout"] = normal(B, L, D)
    else:
        M, K, N = case["M"], case["K"], case["N"]
        s["x"], s["w"] = normal(M, K), normal(N, K, std=K ** -0.5)
        s["b"] = normal(N, dtype=torch.float32, std=0.2) if case["bias"] else None
        s["res"] = normal(M, N) if case["residual"] else None
        if case["do"] == "train":
            s["dout"] = normal(M, N)
    return s


# ---- one pass ----

def run(state):
    if own:
        return _own(state)
    return {"glr": _glr, "gnorm": _gnorm, "linear": _linear}[state["case"]["op"]](state)


def _own(s):
    import selective_state_space_mamba_amd as ms
    c = s["case"]
    if c["op"] == "glr":
        kw = dict(scale=SCALE, input_rule={"sqrt": ms.GLR_SQRT, "lerp": ms.GLR_LERP, "unit": ms.GLR_UNIT}[c["rule"]])
        args = (s["x"], s["r"], s["i"], s["z"], s["lam"])
        if c["do"] == "step":
            return dict(out=ms.glr_step(s["init"], *args, **kw), state=s["init"])
        kw.update(reverse=c["reverse"], reset=s["reset"], initial_state=s["init"])
        if c["do"] == "fwd":
            out, last = ms.glr_fwd(*args, **kw)
            return dict(out=out, last_state=last)
        out, last, saved = ms.glr_fwd_save(*args, **kw)
        grads = ms.glr_bwd(*args, dout=s["dout"], saved=saved, **kw)
        return dict(grads, out=out, last_state=last)
    act = {"none": ms.ACT_NONE, "relu": ms.ACT_RELU, "silu": ms.ACT_SILU, "gelu": ms.ACT_GELU}[c["act"]]
    if c["op"] == "gnorm":
        out, mean, rstd = ms.group_norm_fwd(s["x"], c["G"], s["w"], s["b"], eps=EPS, act=act)
        if c["do"] == "fwd":
            return dict(out=out, mean=mean, rstd=rstd)
        grads = ms.group_norm_bwd(s["x"], c["G"], s["w"], s["b"], dout=s["dout"], mean=mean, rstd=rstd, act=act)
        return dict(grads, out=out, mean=mean, rstd=rstd)
    train = c["do"] == "train"
    out, pre = ms.linear_fwd(s["x"], s["w"], s["b"], s["res"], act=act, want_pre=train and act != ms.ACT_NONE)
    if not train:
        return dict(out=out)
    grads = ms.linear_bwd(s["x"], s["w"], dout=s["dout"], pre=pre, act=act, want_dbias=s["b"] is not None)
    return dict(grads, out=out)


# ---- the plain forms ----

def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _prefix(a, b):
    """h[t] = a[t]·h[t-1] + b[t] along axis 1, from zero: the pairs (a, b) composed over doubled distances."""
    step, n = 1, b.shape[1]
    while step < n:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _glr(s):
    c = s["case"]
    dt = s["x"].dtype
    x, r = s["x"].float(), s["r"].float()
    q = torch.sigmoid(r)
    if s["lam"] is not None:
        rate = SCALE * _softplus(s["lam"])
        e = rate * q
    else:
        e = _softplus(-r)
    a = torch.exp(-e)
    if c["rule"] == "sqrt":
        beta = torch.sqrt(-torch.expm1(-2 * e))
    elif c["rule"] == "lerp":
        beta = -torch.expm1(-e)
    else:
        beta = torch.ones_like(e)
    p = torch.sigmoid(s["i"].float()) if s["i"] is not None else 1.0
    b = beta * (p * x)
    if c["do"] == "step":
        h = a * s["init"] + b
        s["init"].copy_(h)
        if s["z"] is not None:
            z = s["z"].float()
            h = h * (z * torch.sigmoid(z))
        return dict(out=h.to(dt), state=s["init"])
    keep = a
    if s["reset"] is not None:
        keep = torch.where(s["reset"][:, :, None] != 0, 0.0, a)
    flip = (lambda v: v.flip(1)) if c["reverse"] else (lambda v: v)
    keep_o, b_o = flip(keep), flip(b)  # in scan order
    first = torch.cat([b_o[:, :1] + keep_o[:, :1] * s["init"][:, None], b_o[:, 1:]], 1)
    h_o = _prefix(keep_o, first)
    h = flip(h_o)
    if s["z"] is not None:
        z = s["z"].float()
        sz = torch.sigmoid(z)
        out = h * (z * sz)
    else:
        out = h
    ret = dict(out=out.to(dt), last_state=h_o[:, -1].clone())
    if c["do"] == "fwd":
        return ret
    dout = s["dout"].float()
    dh = dout * (z * sz) if s["z"] is not None else dout
    # adjoint: m[t] = dh[t] + keep[t+1]·m[t+1] in scan order
    after = torch.cat([keep_o[:, 1:], torch.zeros_like(keep_o[:, :1])], 1)
    m_o = _prefix(after.flip(1), flip(dh).flip(1)).flip(1)
    m = flip(m_o)
    before = flip(torch.cat([s["init"][:, None], h_o[:, :-1]], 1))
    if c["rule"] == "sqrt":
        dbeta = a * a / torch.clamp(beta, min=1e-18)
    elif c["rule"] == "lerp":
        dbeta = a
    else:
        dbeta = 0.0
    de = m * (p * x * dbeta - keep * before)
    ret["dx"] = (m * beta * p).to(dt)
    if s["lam"] is not None:
        ret["dr"] = (de * e * (1 - q)).to(dt)
        ret["dlam"] = (de * q).sum((0, 1)) * SCALE * torch.sigmoid(s["lam"])
    else:
        ret["dr"] = (-de * torch.sigmoid(-r)).to(dt)
    if s["i"] is not None:
        ret["di"] = (m * beta * x * p * (1 - p)).to(dt)
    if s["z"] is not None:
        ret["dz"] = (dout * h * (sz * (1 + z * (1 - sz)))).to(dt)
    ret["dinit"] = keep_o[:, 0] * m_o[:, 0]
    return ret


def _act(u, act):
    if act == "relu":
        return torch.clamp(u, min=0)
    if act == "silu":
        return u * torch.sigmoid(u)
    if act == "gelu":
        return 0.5 * u * (1 + torch.erf(u * 0.5 ** 0.5))
    return u


def _dact(u, act):
    if act == "relu":
        return (u > 0).to(u.dtype)
    if act == "silu":
        q = torch.sigmoid(u)
        return q * (1 + u * (1 - q))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(u * 0.5 ** 0.5)) + u * torch.exp(-0.5 * u * u) * (2 * math.pi) ** -0.5
    return torch.ones_like(u)


def _gnorm(s):
    c = s["case"]
    B, L, D, G = c["B"], c["L"], c["D"], c["G"]
    x = s["x"].float().view(B, L, G, D // G)
    mean = x.mean((1, 3), keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean((1, 3), keepdim=True) + EPS)
    xh = xc * rstd
    w, b = s["w"].view(G, D // G), s["b"].view(G, D // G)
    u = xh * w + b
    ret = dict(out=_act(u, c["act"]).view(B, L, D).to(s["x"].dtype), mean=mean.view(B, G).clone(),
               rstd=rstd.view(B, G).clone())
    if c["do"] == "fwd":
        return ret
    du = s["dout"].float().view(B, L, G, D // G) * _dact(u, c["act"])
    ret["dweight"], ret["dbias"] = (du * xh).sum((0, 1)).view(D), du.sum((0, 1)).view(D)
    t = du * w
    dx = rstd * (t - t.mean((1, 3), keepdim=True) - xh * (t * xh).mean((1, 3), keepdim=True))
    ret["dx"] = dx.view(B, L, D).to(s["x"].dtype)
    return ret


def _linear(s):
    c = s["case"]
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    u = x @ w.t()
    if s["b"] is not None:
        u = u + s["b"]
    out = _act(u, c["act"])
    if s["res"] is not None:
        out = out + s["res"].float()
    ret = dict(out=out.to(dt))
    if c["do"] == "fwd":
        return ret
    du = s["dout"].float() * _dact(u, c["act"])
    ret["dx"], ret["dweight"] = (du @ w).to(dt), (du.t() @ x).to(dt)
    if s["b"] is not None:
        ret["dbias"] = du.sum(0)
    return ret


# ---- what a pass cannot do without ----

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "glr":
        n, rows = case["B"] * case["L"] * case["D"], case["B"] * case["D"]
        ins = 2 + case["gate"] + case["z"]
        by = e * n * (ins + 1) + 8 * rows + (4 * case["D"] if case["lam"] else 0)
        by += case["B"] * case["L"] if case["reset"] else 0
        fl = n * (14 + 6 * case["gate"] + 6 * case["z"])
        if case["do"] == "train":  # inputs and the upstream gradient again, and every gradient
            by += e * n * (2 * ins + 1) + 4 * rows + (4 * case["D"] if case["lam"] else 0)
            fl += n * (40 + 12 * case["gate"] + 12 * case["z"])
        return {"bytes": by, "flops": fl}
    if case["op"] == "gnorm":
        n = case["B"] * case["L"] * case["D"]
        by, fl = 2 * e * n + 8 * case["D"] + 8 * case["B"] * case["G"], 12 * n
        if case["do"] == "train":
            by, fl = by + 3 * e * n + 8 * case["D"], fl + 24 * n
        return {"bytes": by, "flops": fl}
    M, K, N = case["M"], case["K"], case["N"]
    by = e * (M * K + N * K + M * N * (2 if case["residual"] else 1)) + (4 * N if case["bias"] else 0)
    fl = 2 * M * K * N
    if case["do"] == "train":
        by += e * (2 * M * K + 2 * N * K + M * N) + (4 * N if case["bias"] else 0)
        fl *= 3
    return {"bytes": by, "flops": fl}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if case["op"] == "glr":
        return _exact_glr(case, d, s["reset"])
    if case["op"] == "gnorm":
        return _exact_gnorm(case, d)
    u = torch.matmul(d["x"], d["w"].t().contiguous()) + d.get("b", 0.0)
    y, dy = _exact_act(u, case["act"])
    ret = dict(out=y + d.get("res", 0.0))
    if case["do"] == "train":
        du = d["dout"] * dy
        ret.update(dx=torch.matmul(du, d["w"]), dweight=torch.matmul(du.t().contiguous(), d["x"]))
        if "b" in d:
            ret["dbias"] = du.sum(0)
    return ret


def _exact_act(u, act):
    """The activation and its derivative."""
    if act == "none":
        return u, torch.ones_like(u)
    if act == "relu":
        on = (u > 0).double()
        return u * on, on
    if act == "silu":
        q = 1 / (1 + torch.exp(-u))
        return u * q, q + u * q * (1 - q)
    cdf = torch.special.erfc(-u / math.sqrt(2)) / 2
    return u * cdf, cdf + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)


def _exact_gnorm(case, d):
    B, L, D, G = case["B"], case["L"], case["D"], case["G"]
    C = D // G
    x = d["x"].view(B, L, G, C).permute(0, 2, 1, 3).reshape(B * G, L * C)
    mean = x.sum(1) / (L * C)
    var = ((x - mean[:, None]) ** 2).sum(1) / (L * C)
    rstd = 1 / torch.sqrt(var + EPS)

    def back(v):
        return v.view(B, G, L, C).permute(0, 2, 1, 3).reshape(B, L, D)

    n = back((x - mean[:, None]) * rstd[:, None])
    y, dy = _exact_act(n * d["w"] + d["b"], case["act"])
    ret = dict(out=y, mean=mean.view(B, G), rstd=rstd.view(B, G))
    if case["do"] == "train":
        du = d["dout"] * dy
        ret.update(dweight=(du * n).sum((0, 1)), dbias=du.sum((0, 1)))
        t = (du * d["w"]).view(B, L, G, C).permute(0, 2, 1, 3).reshape(B * G, L * C)
        xh = (x - mean[:, None]) * rstd[:, None]
        m1, m2 = t.sum(1) / (L * C), (t * xh).sum(1) / (L * C)
        ret["dx"] = back(rstd[:, None] * (t - m1[:, None] - xh * m2[:, None]))
    return ret


def _exact_glr(case, d, reset):
    """One position after the other, in scan order."""
    x, r = d["x"], d["r"]
    q = 1 / (1 + torch.exp(-r))
    e = SCALE * torch.log1p(torch.exp(d["lam"])) * q if "lam" in d else torch.log1p(torch.exp(-r))
    a = torch.exp(-e)
    om = {"sqrt": 2.0, "lerp": 1.0, "unit": 0.0}[case["rule"]]
    beta = -torch.expm1(-om * e) if om else torch.ones_like(e)
    if case["rule"] == "sqrt":
        beta = torch.sqrt(beta)
    p = 1 / (1 + torch.exp(-d["i"])) if "i" in d else torch.ones_like(x)
    v = p * x
    if "z" in d:
        sz = 1 / (1 + torch.exp(-d["z"]))
        gate, dgate = d["z"] * sz, sz + d["z"] * sz * (1 - sz)
    else:
        gate = dgate = torch.ones_like(x)
    if case["do"] == "step":
        h = a * d["init"] + beta * v
        return dict(out=h * gate, state=h)
    k = a if reset is None else a * (reset == 0).double()[:, :, None]
    L = case["L"]
    order = range(L - 1, -1, -1) if case["reverse"] else range(L)
    bv = beta * v
    h = torch.empty_like(x)
    prev = d["init"]
    before = torch.empty_like(x) if case["do"] == "train" else None
    for t in order:
        if before is not None:
            before[:, t] = prev
        prev = torch.addcmul(bv[:, t], k[:, t], prev, out=h[:, t])
    ret = dict(out=h * gate, last_state=prev.clone())
    if case["do"] == "fwd":
        return ret
    dh = d["dout"] * gate
    m = torch.empty_like(x)
    carry = torch.zeros_like(prev)
    for t in reversed(order):
        torch.add(dh[:, t], carry, out=m[:, t])
        carry = k[:, t] * m[:, t]
    # dβ/de·de/dr with the factors of the limits e -> 0 kept together
    db = {"sqrt": a * a / torch.clamp(beta, min=1e-150), "lerp": a, "unit": torch.zeros_like(a)}[case["rule"]]
    de = m * (v * db - k * before)
    ret["dx"] = m * beta * p
    if "lam" in d:
        ret["dr"] = de * e * (1 - q)
        ret["dlam"] = (de * q).sum((0, 1)) * SCALE / (1 + torch.exp(-d["lam"]))
    else:
        ret["dr"] = -de / (1 + torch.exp(r))
    if "i" in d:
        ret["di"] = m * beta * x * p * (1 - p)
    if "z" in d:
        ret["dz"] = d["dout"] * h * dgate
    ret["dinit"] = carry
    return ret

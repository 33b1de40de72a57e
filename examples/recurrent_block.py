"""A residual block around the gated linear recurrence, made of the library's
operators alone: per-head normalisation of every token, four projections,
the recurrence with its gates, and the projection back onto the residual stream.

    n = group_norm(x)                    (every token by itself, G heads)
    p, r, i, z = n·W_kᵀ + b_k
    h = glr(p, r, i, z, lam)
    y = h·W_oᵀ + b_o + x

forward() and backward() run whole sequences, step() one token of each sequence
from the recurrent state.  Run it to train a block on a toy task (recall the
input of two tokens before) and to check the token-by-token path against the
whole-sequence one:

    python examples/recurrent_block.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import selective_state_space_mamba_amd as ms  # noqa: E402

GATES = ("p", "r", "i", "z")


class RecurrentBlock:
    def __init__(self, dim, inner, groups, dtype=torch.bfloat16, device="cuda:0", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std

        self.dim, self.groups, self.dtype = dim, groups, dtype
        w = {"w_" + k: normal(inner, dim, std=dim ** -0.5).to(dtype) for k in GATES}
        w["w_o"] = normal(dim, inner, std=inner ** -0.5).to(dtype)
        w.update({"b_" + k: torch.zeros(inner, device=device) for k in GATES}, b_o=torch.zeros(dim, device=device))
        a = 0.6 + 0.39 * torch.rand(inner, generator=g, device=device)  # decays at an open gate
        w["lam"] = torch.log(torch.expm1(-torch.log(a) / 8.0))
        w.update(norm_w=torch.ones(dim, device=device), norm_b=torch.zeros(dim, device=device))
        self.w = w

    def _norm(self, x):
        n, mean, rstd = ms.group_norm_fwd(x.view(-1, 1, self.dim), self.groups, self.w["norm_w"], self.w["norm_b"])
        return n.view(x.shape), mean, rstd

    def _project(self, n):
        return {k: ms.linear_fwd(n, self.w["w_" + k], self.w["b_" + k])[0] for k in GATES}

    def forward(self, x, state=None, reset=None):
        """x [B][L][dim]; returns (y, last_state) and keeps what backward() needs."""
        n, mean, rstd = self._norm(x)
        g = self._project(n)
        h, last, saved = ms.glr_fwd_save(g["p"], g["r"], g["i"], g["z"], self.w["lam"], initial_state=state,
                                         reset=reset)
        y, _ = ms.linear_fwd(h, self.w["w_o"], self.w["b_o"], x)
        self.kept = (x, n, mean, rstd, g, h, saved, state, reset)
        return y, last

    def backward(self, dy):
        """Gradients for dy [B][L][dim]: (dx, {name: gradient})."""
        x, n, mean, rstd, g, h, saved, state, reset = self.kept
        out = ms.linear_bwd(h, self.w["w_o"], dout=dy)
        grads = dict(w_o=out["dweight"], b_o=out["dbias"])
        d = ms.glr_bwd(g["p"], g["r"], g["i"], g["z"], self.w["lam"], dout=out["dx"], initial_state=state,
                       reset=reset, saved=saved)
        grads["lam"] = d["dlam"]
        dn = 0.0
        for k, name in zip(GATES, ("dx", "dr", "di", "dz")):
            one = ms.linear_bwd(n, self.w["w_" + k], dout=d[name])
            grads["w_" + k], grads["b_" + k] = one["dweight"], one["dbias"]
            dn = dn + one["dx"].float()
        norm = ms.group_norm_bwd(x.view(-1, 1, self.dim), self.groups, self.w["norm_w"], self.w["norm_b"],
                                 dout=dn.to(self.dtype).view(-1, 1, self.dim), mean=mean, rstd=rstd)
        grads["norm_w"], grads["norm_b"] = norm["dweight"], norm["dbias"]
        return norm["dx"].view(x.shape) + dy, grads

    def step(self, x_t, state):
        """One token a sequence: x_t [B][dim], state [B][inner] float32, updated in place.  Returns y_t."""
        n, _, _ = self._norm(x_t)
        g = self._project(n)
        h = ms.glr_step(state, g["p"], g["r"], g["i"], g["z"], self.w["lam"])
        return ms.linear_fwd(h, self.w["w_o"], self.w["b_o"], x_t)[0]


def main(steps=60):
    B, L, D = 8, 192, 128
    block = RecurrentBlock(D, 256, 4)
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(1)
    master = {k: v.float() for k, v in block.w.items()}
    m1 = {k: torch.zeros_like(v) for k, v in master.items()}
    m2 = {k: torch.zeros_like(v) for k, v in master.items()}
    losses = []
    for it in range(steps):
        x = torch.randn(B, L, D, generator=gen, device="cuda:0").to(block.dtype)
        y, _ = block.forward(x)
        err = y.float()[:, 2:] - x.float()[:, :-2]
        losses.append(float((err * err).mean()))
        dy = torch.zeros(B, L, D, device="cuda:0")
        dy[:, 2:] = 2.0 * err / err.numel()
        _, grads = block.backward(dy.to(block.dtype))
        for k, g in grads.items():
            g = g.float()
            m1[k] = 0.9 * m1[k] + 0.1 * g
            m2[k] = 0.99 * m2[k] + 0.01 * g * g
            upd = (m1[k] / (1 - 0.9 ** (it + 1))) / ((m2[k] / (1 - 0.99 ** (it + 1))).sqrt() + 1e-12)
            master[k] -= 3e-3 * upd
            block.w[k] = master[k].to(block.w[k].dtype)
    print("recall loss: %.3f at the start, %.3f after %d steps" % (losses[0], losses[-1], steps))
    x = torch.randn(B, L, D, generator=gen, device="cuda:0").to(block.dtype)
    y, last = block.forward(x)
    state = torch.zeros_like(last)
    tokens = torch.stack([block.step(x[:, t].contiguous(), state) for t in range(L)], 1)
    off = float((tokens.float() - y.float()).abs().max() / y.float().abs().max())
    print("token by token against whole sequences: %.1e of the largest output" % off)
    return losses, off


if __name__ == "__main__":
    main()

"""The layer operators (short causal convolution, selective state space scan, group norm,
projection) from their definitions, in float64 torch on any device, step by step. Gradients come
from autograd through these definitions."""
from __future__ import annotations

import torch


def act(name, x):
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return x * torch.special.ndtr(x)
    return x


def conv(x, w, bias, s0, lens, name):
    """(y, s_T), looping over the taps of each row's valid steps."""
    B, T, C = x.shape
    W = w.shape[1]
    ys, states = [], []
    for b in range(B):
        L = T if lens is None else min(max(int(lens[b]), 0), T)
        head = x.new_zeros(W - 1, C) if s0 is None else s0[b]
        rows = torch.cat([head, x[b, :L]])
        pre = x.new_zeros(L, C) if bias is None else bias.expand(L, C)
        for j in range(W):
            pre = pre + w[:, j] * rows[j:j + L]
        ys.append(torch.cat([act(name, pre), x.new_zeros(T - L, C)]))
        states.append(rows[L:])
    return torch.stack(ys), torch.stack(states)


def scan(u, dt, A_log, B, C, D, dt_bias, z, h0, lens):
    """(y, h_T), one step at a time."""
    Bn, T, Cn = u.shape
    G, N = B.shape[2:]
    A = -torch.exp(A_log)
    raw = dt if dt_bias is None else dt + dt_bias
    d = torch.nn.functional.softplus(raw, threshold=40.0)
    h = u.new_zeros(Bn, Cn, N) if h0 is None else h0
    n = torch.full((Bn,), T, device=u.device) if lens is None else lens.clamp(0, T)
    ys = []
    for t in range(T):
        on = (t < n)[:, None]
        Bt = B[:, t].repeat_interleave(Cn // G, 1)
        Ct = C[:, t].repeat_interleave(Cn // G, 1)
        new = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * u[:, t])[..., None] * Bt
        h = torch.where(on[..., None], new, h)
        y = (h * Ct).sum(-1)
        if D is not None:
            y = y + D * u[:, t]
        if z is not None:
            y = y * act("silu", z[:, t])
        ys.append(torch.where(on, y, torch.zeros_like(y)))
    return torch.stack(ys, 1), h


def norm(x, groups, w, b, z, name, eps, center):
    C = x.shape[-1]
    g = x.reshape(*x.shape[:-1], groups, C // groups)
    if center:
        g = g - g.mean(-1, keepdim=True)
    xh = (g / torch.sqrt((g * g).mean(-1, keepdim=True) + eps)).reshape(x.shape)
    aff = xh if w is None else xh * w
    aff = aff if b is None else aff + b
    return act(name, aff) if z is None else aff * act(name, z)


def linear(x, W, bias, res, name):
    pre = x @ W.t()
    if bias is not None:
        pre = pre + bias
    y = act(name, pre)
    return y if res is None else y + res


def with_grads(f, leaves, cotangents):
    """f(**leaves) -> tensor or tuple, and the gradients of sum <cotangent, output> by autograd: a
    dict over the leaves that are not None."""
    live = {k: v.detach().clone().requires_grad_(True) for k, v in leaves.items() if v is not None}
    out = f(**{k: live.get(k) for k in leaves})
    outs = out if isinstance(out, tuple) else (out,)
    loss = sum((o * c).sum() for o, c in zip(outs, cotangents) if c is not None)
    grads = torch.autograd.grad(loss, list(live.values()), allow_unused=True)
    grads = {k: torch.zeros_like(live[k]) if g is None else g for k, g in zip(live, grads)}
    return tuple(o.detach() for o in outs), grads


def rel(got, ref):
    """Relative 2-norm error; infinite where the finite places differ."""
    got, ref = got.detach().double(), ref.detach().double()
    if got.shape != ref.shape or not torch.equal(torch.isfinite(got), torch.isfinite(ref)):
        return float("inf")
    ok = torch.isfinite(ref)
    d, n = torch.linalg.vector_norm((got - ref)[ok]).item(), torch.linalg.vector_norm(ref[ok]).item()
    return d / n if n > 0 else (0.0 if d == 0 else float("inf"))

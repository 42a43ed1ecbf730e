"""Linear attention with a decay and the norms around a block from their definitions, in float64 torch on
any device, step by step. Gradients come from autograd through these definitions."""
from __future__ import annotations

import torch

import layer_reference as R


def linattn(q, k, v, g, S0, lens):
    """(y, S_T), one step at a time; gradients reach q, k, v and S0."""
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    own = torch.arange(Hv, device=q.device) // (Hv // Hk)
    n = torch.full((B,), T, device=q.device) if lens is None else lens.clamp(0, T)
    ok = (torch.arange(T, device=q.device) < n[:, None])[:, :, None, None]
    q, k, v = (torch.where(ok, t, 0.0) for t in (q, k, v))            # what lies behind a row is not read
    S = q.new_zeros(B, Hv, Dv, Dk) if S0 is None else S0
    ys = []
    for t in range(T):
        on = (t < n)[:, None, None, None]
        new = g.to(q.dtype)[:, None, None] * S + v[:, t, :, :, None] * k[:, t, own][:, :, None]
        S = torch.where(on, new, S)
        ys.append(torch.where(on[..., 0], (S * q[:, t, own][:, :, None]).sum(-1), 0.0))
    return torch.stack(ys, 1), S


def resnorm(x, h, z, scale, w_post, w_pre, post, pre, act, eps):
    """(r, y)"""
    rms = lambda t: torch.sqrt((t * t).mean(-1, keepdim=True) + eps)  # noqa: E731
    n = h / rms(h) if post else h
    n = n if w_post is None else n * w_post
    if z is not None:
        gate = R.act(act, z)
        while gate.dim() < x.dim():
            gate = gate.unsqueeze(-2)
        n = n * gate
    r = x + (n if scale is None else n * scale)
    if not pre:
        return (r,)
    y = r / rms(r)
    return r, (y if w_pre is None else y * w_pre)

"""Recurrent layers built from the library's calls, as a model would run them: a gated delta rule layer, a
selective scan layer and blocks of linear attention on a residual stream, each for prompts, single
tokens (state carried and updated in place) and training steps (forward and backward).

    python examples/recurrent_layers.py

prints, for each of them, how far a prompt continued token by token is from one long prompt, and the
time of a prompt, a token and a training step. PyTorch holds the tensors; every operation on them
other than slicing, copying and adding gradients is a call of the library.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_22_gb300 as gdn  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def _normal(gen, *shape, scale=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


class GatedDeltaLayer:
    """x -> projection -> short convolution of q, k, v -> unit q and k, gates -> gated delta rule -> head
    norm gated by z -> projection + x."""

    def __init__(self, width=512, Hk=2, Hv=4, Dk=64, Dv=64, taps=4, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.Hk, self.Hv, self.Dk, self.Dv = Hk, Hv, Dk, Dv
        self.nk, self.nv = Hk * Dk, Hv * Dv
        # q | k | v | z | a | b, each padded to whole 16 bytes
        self.cuts = [0, self.nk, 2 * self.nk, 2 * self.nk + self.nv, 2 * (self.nk + self.nv)]
        self.cuts += [self.cuts[4] + (Hv + 7) // 8 * 8]
        out = self.cuts[5] + (Hv + 7) // 8 * 8
        self.W_in = _normal(gen, out, width, scale=width ** -0.5)
        self.W_out = _normal(gen, width, self.nv, scale=self.nv ** -0.5)
        self.taps = [_normal(gen, n, taps, scale=taps ** -0.5, dtype=F32) for n in (self.nk, self.nk, self.nv)]
        self.A_log, self.dt_bias = _normal(gen, Hv, scale=0.5, dtype=F32), _normal(gen, Hv, scale=0.5, dtype=F32)
        self.w = torch.ones(self.nv, device="cuda")
        self.w_q = torch.full((self.nk,), 1.0 / Dk, device="cuda")      # rms norm / sqrt(Dk) is a unit vector; q / sqrt(Dk) too
        self.w_k = torch.full((self.nk,), Dk ** -0.5, device="cuda")

    def start(self, B):
        W = self.taps[0].shape[1]
        conv = [torch.zeros(B, W - 1, n, device="cuda", dtype=BF16) for n in (self.nk, self.nk, self.nv)]
        return {"conv": conv, "S": torch.zeros(B, self.Hv, self.Dv, self.Dk, device="cuda")}

    def _split(self, p):
        c = self.cuts
        q, k, v, z = (p[..., c[i]:c[i + 1]] for i in range(4))
        return q, k, v, z, p[..., c[4]:c[4] + self.Hv].contiguous(), p[..., c[5]:c[5] + self.Hv].contiguous()

    def forward(self, x, state=None, train=False):
        """y and the state behind x (updated in place for one token); train: y and what backward needs."""
        B, T, _ = x.shape
        s = self.start(B) if state is None else state
        p, _ = gdn.gdn_linear_fwd(x, self.W_in)
        q, k, v, z, a, b = self._split(p)
        conv, ends = [], []
        for t, w, s0 in zip((q, k, v), self.taps, s["conv"]):
            y, end = gdn.gdn_conv_fwd(t, w, None, s0, s_T=s0 if T == 1 else None)
            conv.append(y)
            ends.append(end)
        qn, q_stats = gdn.gdn_norm_fwd(conv[0], self.Hk, self.w_q, act="none", center=False, eps=1e-6)
        kn, k_stats = gdn.gdn_norm_fwd(conv[1], self.Hk, self.w_k, act="none", center=False, eps=1e-6)
        q4, k4 = qn.view(B, T, self.Hk, self.Dk), kn.view(B, T, self.Hk, self.Dk)
        v4 = conv[2].view(B, T, self.Hv, self.Dv)
        g, beta = gdn.gdn_gates_fwd(a, b, self.A_log, self.dt_bias, Hk=self.Hk, Dk=self.Dk, Dv=self.Dv)
        ck = None
        if train:
            o, S, ck = gdn.gdn_fwd(q4, k4, v4, g, beta, s["S"])
        elif T == 1:
            o, S, _ = gdn.gdn_fwd(q4, k4, v4, g, beta, s["S"], S_T=s["S"], want_ckpt=False)
        else:
            o, S = gdn.gdn_fwd_infer(q4, k4, v4, g, beta, s["S"])
        o = o.view(B, T, self.nv)
        n, stats = gdn.gdn_norm_fwd(o, self.Hv, self.w, None, z, act="silu", center=False)
        y, _ = gdn.gdn_linear_fwd(n, self.W_out, None, x)
        if not train:
            return y, {"conv": ends, "S": S}
        return y, dict(x=x, p=p, s=s, conv=conv, q_stats=q_stats, k_stats=k_stats, q4=q4, k4=k4, v4=v4, g=g, beta=beta, ck=ck, o=o,
                       n=n, stats=stats)

    def backward(self, c, dy):
        """Gradients of x and of the parameters for the cotangent dy of y."""
        B, T, _ = dy.shape
        q, k, v, z, a, b = self._split(c["p"])
        out = gdn.gdn_linear_bwd(c["n"], self.W_out, dy, want_dbias=False)
        nb = gdn.gdn_norm_bwd(c["o"], self.Hv, c["stats"], out["dx"], self.w, None, z, act="silu", center=False)
        r = gdn.gdn_bwd(c["q4"], c["k4"], c["v4"], c["g"], c["beta"], c["ck"], nb["dx"].view(B, T, self.Hv, self.Dv))
        ga = gdn.gdn_gates_bwd(a, b, self.A_log, self.dt_bias, r["dg"], r["dbeta"], Hk=self.Hk, Dk=self.Dk, Dv=self.Dv)
        dq = gdn.gdn_norm_bwd(c["conv"][0], self.Hk, c["q_stats"], r["dq"].view(B, T, self.nk), self.w_q, act="none", center=False)["dx"]
        dk = gdn.gdn_norm_bwd(c["conv"][1], self.Hk, c["k_stats"], r["dk"].view(B, T, self.nk), self.w_k, act="none", center=False)["dx"]
        dp = torch.zeros_like(c["p"])
        taps = []
        for i, (t, w, s0, d) in enumerate(zip((q, k, v), self.taps, c["s"]["conv"], (dq, dk, r["dv"].view(B, T, self.nv)))):
            cb = gdn.gdn_conv_bwd(t, w, d, None, s0, want_ds0=False)
            dp[..., self.cuts[i]:self.cuts[i + 1]] = cb["dx"]
            taps.append(cb["dw"])
        dp[..., self.cuts[3]:self.cuts[4]] = nb["dz"]
        dp[..., self.cuts[4]:self.cuts[4] + self.Hv] = ga["da"]
        dp[..., self.cuts[5]:self.cuts[5] + self.Hv] = ga["db"]
        inp = gdn.gdn_linear_bwd(c["x"], self.W_in, dp, want_dbias=False)
        return {"dx": inp["dx"] + dy, "dW_in": inp["dW"], "dW_out": out["dW"], "dtaps": taps, "dA_log": ga["dA_log"],
                "ddt_bias": ga["ddt_bias"], "dw": nb["dw"]}


class SelectiveScanLayer:
    """x -> projection to u and z -> short convolution -> projection to the low-rank step, B and C ->
    selective scan gated by z -> projection + x."""

    def __init__(self, width=512, channels=1024, states=16, rank=32, taps=4, seed=1):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.C, self.N, self.R = channels, states, rank
        self.W_in = _normal(gen, 2 * channels, width, scale=width ** -0.5)
        self.taps, self.bias = _normal(gen, channels, taps, scale=taps ** -0.5, dtype=F32), torch.zeros(channels, device="cuda")
        self.W_x = _normal(gen, rank + 2 * states, channels, scale=channels ** -0.5)
        self.W_dt = _normal(gen, channels, rank, scale=rank ** -0.5)
        self.A_log = torch.log(torch.arange(1, states + 1, device="cuda", dtype=F32)).repeat(channels, 1)
        step = torch.exp(torch.rand(channels, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
        self.dt_bias = step + torch.log(-torch.expm1(-step))
        self.D = torch.ones(channels, device="cuda")
        self.W_out = _normal(gen, width, channels, scale=channels ** -0.5)

    def start(self, B):
        return {"conv": torch.zeros(B, self.taps.shape[1] - 1, self.C, device="cuda", dtype=BF16),
                "h": torch.zeros(B, self.C, self.N, device="cuda")}

    def _scan_inputs(self, r, u, dt, z):
        B, T, _ = u.shape
        Bm = r[..., self.R:self.R + self.N].unflatten(-1, (1, self.N))
        Cm = r[..., self.R + self.N:].unflatten(-1, (1, self.N))
        return u, dt, self.A_log, Bm, Cm, self.D, self.dt_bias, z

    def forward(self, x, state=None, train=False, lens=None):
        B, T, _ = x.shape
        s = self.start(B) if state is None else state
        p, _ = gdn.gdn_linear_fwd(x, self.W_in)
        u_in, z = p[..., :self.C], p[..., self.C:]
        u, end = gdn.gdn_conv_fwd(u_in, self.taps, self.bias, s["conv"], lens, s_T=s["conv"] if T == 1 else None)
        r, _ = gdn.gdn_linear_fwd(u, self.W_x)
        dt, _ = gdn.gdn_linear_fwd(r[..., :self.R], self.W_dt)
        y, h, ck = gdn.gdn_scan_fwd(*self._scan_inputs(r, u, dt, z), s["h"], lens, h_T=s["h"] if T == 1 and not train else None,
                                    want_ckpt=train)
        out, _ = gdn.gdn_linear_fwd(y, self.W_out, None, x)
        if not train:
            return out, {"conv": end, "h": h}
        return out, dict(x=x, p=p, s=s, u=u, r=r, dt=dt, y=y, ck=ck, lens=lens)

    def backward(self, c, dy):
        u_in, z = c["p"][..., :self.C], c["p"][..., self.C:]
        out = gdn.gdn_linear_bwd(c["y"], self.W_out, dy, want_dbias=False)
        u, dt, A_log, Bm, Cm, D, dt_bias, z = self._scan_inputs(c["r"], c["u"], c["dt"], z)
        sc = gdn.gdn_scan_bwd(u, dt, A_log, Bm, Cm, c["ck"], out["dx"], D, dt_bias, z, c["lens"], want_dh0=False)
        step = gdn.gdn_linear_bwd(c["r"][..., :self.R], self.W_dt, sc["ddt"], want_dbias=False)
        dr = torch.cat([step["dx"], sc["dB"].flatten(-2), sc["dC"].flatten(-2)], -1)
        mid = gdn.gdn_linear_bwd(c["u"], self.W_x, dr, want_dbias=False)
        cb = gdn.gdn_conv_bwd(u_in, self.taps, sc["du"] + mid["dx"], self.bias, c["s"]["conv"], c["lens"], want_ds0=False)
        inp = gdn.gdn_linear_bwd(c["x"], self.W_in, torch.cat([cb["dx"], sc["dz"]], -1), want_dbias=False)
        return {"dx": inp["dx"] + dy, "dW_in": inp["dW"], "dW_x": mid["dW"], "dW_dt": step["dW"], "dW_out": out["dW"],
                "dtaps": cb["dw"], "dbias": cb["dbias"], "dA_log": sc["dA_log"], "dD": sc["dD"], "ddt_bias": sc["ddt_bias"]}


class LinearAttentionBlocks:
    """Blocks on a residual stream: norm -> projection to q, k, v and z -> linear attention with a decay for
    each head -> head norm gated by z -> projection -> norm, residual scale and addition onto the stream,
    with the norm in front of the next block. Returns the stream's norm behind the last block."""

    def __init__(self, width=512, Hk=2, Hv=4, Dk=64, Dv=64, blocks=2, seed=3):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.Hk, self.Hv, self.Dk, self.Dv, self.width = Hk, Hv, Dk, Dv, width
        self.nk, self.nv = Hk * Dk, Hv * Dv
        around = lambda n, mean: mean + _normal(gen, n, scale=0.1, dtype=F32)  # noqa: E731
        self.g = torch.exp(-torch.exp2(-8.0 * torch.arange(1, Hv + 1, device="cuda") / Hv))
        self.w_first = around(width, 1.0)
        self.blocks = []
        for _ in range(blocks):
            W_in = _normal(gen, 2 * (self.nk + self.nv), width, scale=width ** -0.5, dtype=F32)
            W_in[:self.nk] *= Dk ** -0.5
            self.blocks.append(dict(W_in=W_in.to(BF16), w_head=around(self.nv, 1.0), W_out=_normal(gen, width, self.nv, scale=self.nv ** -0.5),
                                    scale=around(width, 0.5), w_post=around(width, 1.0), w_pre=around(width, 1.0)))

    def start(self, B):
        return [torch.zeros(B, self.Hv, self.Dv, self.Dk, device="cuda") for _ in self.blocks]

    def _split(self, p):
        a, b, c = self.nk, 2 * self.nk, 2 * self.nk + self.nv
        return (p[..., :a].unflatten(-1, (self.Hk, self.Dk)), p[..., a:b].unflatten(-1, (self.Hk, self.Dk)),
                p[..., b:c].unflatten(-1, (self.Hv, self.Dv)), p[..., c:])

    def forward(self, x, state=None, train=False, lens=None):
        B, T, _ = x.shape
        states = self.start(B) if state is None else state
        n, first_stats = gdn.gdn_norm_fwd(x, 1, self.w_first, act="none", center=False)
        ends, kept, first = [], [], x
        for w, S0 in zip(self.blocks, states):
            p, _ = gdn.gdn_linear_fwd(n, w["W_in"])
            q, k, v, z = self._split(p)
            o, S = gdn.gdn_linattn_fwd(q, k, v, self.g, S0, lens, S_T=S0 if T == 1 and not train else None)
            o = o.view(B, T, self.nv)
            m, head_stats = gdn.gdn_norm_fwd(o, self.Hv, w["w_head"], None, z, act="silu", center=False)
            h, _ = gdn.gdn_linear_fwd(m, w["W_out"])
            r, y, stats = gdn.gdn_resnorm_fwd(x, h, None, w["scale"], w["w_post"], w["w_pre"])
            kept.append(dict(n=n, p=p, S0=S0, o=o, m=m, head_stats=head_stats, h=h, x=x, stats=stats))
            ends.append(S)
            x, n = r, y
        return n, (dict(blocks=kept, x=first, first_stats=first_stats, lens=lens) if train else ends)

    def backward(self, c, dy):
        """Gradients of x and of the parameters for the cotangent dy of what forward returns."""
        dn, dx, grads = dy, None, []
        for w, s in zip(reversed(self.blocks), reversed(c["blocks"])):
            B, T, _ = dn.shape
            rb = gdn.gdn_resnorm_bwd(s["x"], s["h"], s["stats"], dn, dx, None, w["scale"], w["w_post"], w["w_pre"])
            out = gdn.gdn_linear_bwd(s["m"], w["W_out"], rb["dh"], want_dbias=False)
            q, k, v, z = self._split(s["p"])
            nb = gdn.gdn_norm_bwd(s["o"], self.Hv, s["head_stats"], out["dx"], w["w_head"], None, z, act="silu", center=False)
            a = gdn.gdn_linattn_bwd(q, k, v, self.g, nb["dx"].view(B, T, self.Hv, self.Dv), s["S0"], c["lens"], want_dS0=False)
            dp = torch.cat([a["dq"].flatten(-2), a["dk"].flatten(-2), a["dv"].flatten(-2), nb["dz"]], -1)
            inp = gdn.gdn_linear_bwd(s["n"], w["W_in"], dp, want_dbias=False)
            grads.insert(0, dict(W_in=inp["dW"], w_head=nb["dw"], W_out=out["dW"], scale=rb["dscale"], w_post=rb["dw_post"], w_pre=rb["dw_pre"]))
            dn, dx = inp["dx"], rb["dx"]
        first = gdn.gdn_norm_bwd(c["x"], 1, c["first_stats"], dn, self.w_first, act="none", center=False)
        return {"dx": dx + first["dx"], "dw_first": first["dw"], "blocks": grads}


def continued(layer, x, tokens):
    """The outputs of x with its last `tokens` steps taken one at a time behind the prompt."""
    T = x.shape[1]
    y, state = layer.forward(x[:, :T - tokens].contiguous())
    ys = [y]
    for t in range(T - tokens, T):
        y, state = layer.forward(x[:, t:t + 1].contiguous(), state)
        ys.append(y)
    return torch.cat(ys, 1)


def _time_us(f, reps=20):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / reps * 1e3


def main():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    for layer in (GatedDeltaLayer(), SelectiveScanLayer(), LinearAttentionBlocks()):
        x = _normal(gen, 2, 260, 512)
        whole, _ = layer.forward(x)
        off = (continued(layer, x, 4).double() - whole.double()).norm() / whole.double().norm()
        long, dy = _normal(gen, 4, 2048, 512), _normal(gen, 4, 2048, 512)
        one, state = _normal(gen, 64, 1, 512), layer.start(64)
        print(f"{type(layer).__name__}: token by token differs by {off.item():.1e} (relative 2-norm); "
              f"prompt 4 x 2048 {_time_us(lambda: layer.forward(long)):.0f} us, "
              f"64 tokens {_time_us(lambda: layer.forward(one, state)):.0f} us, "
              f"training step 4 x 2048 {_time_us(lambda: layer.backward(layer.forward(long, train=True)[1], dy)):.0f} us")


if __name__ == "__main__":
    main()

"""The operators around the gated delta rule in a recurrent layer, as measured cases.

A recurrent layer runs a projection (matrix product with bias and activation), a short causal
convolution over the projected channels, a recurrence (the gated delta rule, or the selective
state space scan measured here), a group norm with a gate, and a projection back onto the
residual stream. The cases below run the four that stand beside the gated delta rule, for
single tokens (serving), prompts (serving) and training steps (forward and backward).

`own = False` computes each operator in its plain form: elementary torch operations in 32 bits,
rounded once at the end. `own = True` calls the library.

    conv    pre[t] = bias + sum_j w[:, j] x[t - W + 1 + j],  y = silu(pre);  x before the first step
            comes from the carried state (the W - 1 newest inputs)
    scan    d = softplus(dt + dt_bias), A = -exp(A_log), h[t] = exp(d A) h[t-1] + d u B,
            y = (C . h + D u) silu(z)
    norm    per row and group: xh = (x - mean) / sqrt(var + eps), y = (xh w + b) silu(z)
    linear  y = act(x W^T + bias) + res
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One generated token for each of 64 sequences: the convolution over the q, k and v channels
        # of the batched layer (16 kv heads and 32 value heads of 128), its state updated.
        dict(name="conv-token", op="conv", dtype="bf16", B=64, T=1, C=8192, W=4, state=True, ragged=False, train=False),
        # Four prompts of different lengths, padded to the longest, that continue a cached prefix.
        dict(name="conv-prompt", op="conv", dtype="bf16", B=4, T=2048, C=8192, W=4, state=True, ragged=True, train=False),
        # A training step's share of the batched layer: forward and backward over 8 x 4096 steps.
        dict(name="conv-train", op="conv", dtype="bf16", B=8, T=4096, C=8192, W=4, state=False, ragged=False, train=True),
        # One generated token for each of 64 sequences: the state is read and written once.
        dict(name="scan-token", op="scan", dtype="bf16", B=64, T=1, C=4096, N=16, G=1, state=True, ragged=False, train=False),
        # One long prompt into an empty cache.
        dict(name="scan-prompt", op="scan", dtype="bf16", B=1, T=4096, C=4096, N=16, G=1, state=False, ragged=False, train=False),
        # A training step: forward and backward.
        dict(name="scan-train", op="scan", dtype="bf16", B=2, T=2048, C=4096, N=16, G=1, state=False, ragged=False, train=True),
        # Training in 32 bits on short ragged rows, odd sizes, two groups of B and C, a carried state.
        dict(name="scan-train-odd", op="scan", dtype="f32", B=3, T=333, C=518, N=11, G=2, state=True, ragged=True, train=True),
        # The head norm and gate behind the recurrence for 64 generated tokens: 32 heads of 128.
        dict(name="norm-token", op="norm", dtype="bf16", M=64, G=32, D=128, gate=True, train=False),
        # The same in a training step over 8 x 4096 steps: forward and backward.
        dict(name="norm-train", op="norm", dtype="bf16", M=32768, G=32, D=128, gate=True, train=True),
        # The input projection of 16 generated tokens: the weights are read once.
        dict(name="linear-token", op="linear", dtype="bf16", M=16, N=8192, K=2048, act="silu", res=False, train=False),
        # The output projection of 8192 prompt tokens onto the residual stream.
        dict(name="linear-prompt", op="linear", dtype="bf16", M=8192, N=2048, K=8192, act="none", res=True, train=False),
        # A projection with an activation in a training step, of sizes that fill no tile: forward and backward.
        dict(name="linear-train", op="linear", dtype="bf16", M=4100, N=2056, K=2040, act="gelu", res=True, train=True),
    ]


def _log_size(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _channels(rng, low, high):
    """A number of channels: any, or (half of the time) a multiple of 64."""
    n = _log_size(rng, low, high)
    if rng.random() < 0.5:
        n = max(64, n // 64 * 64)
    return n + 64 if n == 3072 else n


def draw(rng):
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    kind = rng.choice(["conv-token", "conv-prompt", "conv-train", "scan-token", "scan-prompt", "scan-train",
                       "norm-token", "norm-train", "linear-token", "linear-prompt", "linear-train"])
    op, use = kind.split("-")
    train = use == "train"
    if op == "conv":
        C = _channels(rng, 96, 8192)
        T = 1 if use == "token" else _log_size(rng, 2, 4096)
        B = _log_size(rng, 1, 128) if use == "token" else rng.randint(1, 8)
        return dict(op=op, dtype=dtype, B=B, T=T, C=C, W=rng.randint(2, 4), state=use == "token" or rng.random() < 0.5,
                    ragged=use != "token" and rng.random() < 0.4, train=train)
    if op == "scan":
        G = rng.choice([1, 1, 2, 4])
        C = max(1, _channels(rng, 64, 4096) // G) * G
        C = C + G * 64 if C == 3072 else C
        N = rng.choice([8, 16, 16, rng.randint(1, 16)])
        T = 1 if use == "token" else _log_size(rng, 2, 4096)
        B = _log_size(rng, 1, 64) if use == "token" else rng.randint(1, max(1, min(8, 4096 // T)))
        return dict(op=op, dtype=dtype, B=B, T=T, C=C, N=N, G=G, state=use == "token" or rng.random() < 0.5,
                    ragged=use != "token" and rng.random() < 0.4, train=train)
    if op == "norm":
        M = _log_size(rng, 1, 128) if use == "token" else _log_size(rng, 128, 32768)
        D = rng.choice([64, 128, 192, 256, rng.randint(24, 256)])
        return dict(op=op, dtype=dtype, M=M, G=rng.randint(1, max(1, 4096 // D)), D=D, gate=rng.random() < 0.7, train=train)
    N, K = _channels(rng, 192, 8192), _channels(rng, 192, 8192)
    if use == "token":
        M = rng.randint(1, 32)
    else:
        M = _log_size(rng, 64, 8192)
        while M * N * K > 8192 * 2048 * 8192 // (3 if train else 1):
            M = max(1, M // 2)
    return dict(op=op, dtype=dtype, M=M, N=N, K=K, act=rng.choice(["none", "silu", "gelu"]), res=rng.random() < 0.5, train=train)


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    def uniform(low, high, *shape):
        return torch.rand(*shape, generator=gen, device="cuda") * (high - low) + low

    s = {"case": case}
    if case["op"] in ("conv", "scan"):
        B, T, C = case["B"], case["T"], case["C"]
        s["lens"] = None
        if case["ragged"]:  # one row is full, one has no valid step at all, the rest lie between
            lens = torch.randint(1, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
            lens[0] = T
            if B > 2:
                lens[B - 1] = 0
            s["lens"] = lens
    if case["op"] == "conv":
        W = case["W"]
        s["x"] = normal(B, T, C)
        s["w"] = uniform(-1.0, 1.0, C, W) / math.sqrt(W)
        s["bias"] = uniform(-0.5, 0.5, C)
        s["s0"] = normal(B, W - 1, C) if case["state"] else None
        if case["train"]:
            s["dy"] = normal(B, T, C)
    elif case["op"] == "scan":
        N, G = case["N"], case["G"]
        s["u"], s["z"] = normal(B, T, C), normal(B, T, C)
        s["dt"] = normal(B, T, C, scale=0.5)
        s["B"], s["C"] = normal(B, T, G, N), normal(B, T, G, N)
        s["A_log"] = torch.log(torch.arange(1, N + 1, device="cuda", dtype=torch.float32)).repeat(C, 1) + uniform(-0.1, 0.1, C, N)
        s["D"] = 1.0 + uniform(-0.1, 0.1, C)
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), C))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(dt_bias) = step
        s["h0"] = torch.randn(B, C, N, generator=gen, device="cuda") * 0.5 if case["state"] else None
        if case["train"]:
            s["dy"] = normal(B, T, C)
    elif case["op"] == "norm":
        M, G, D = case["M"], case["G"], case["D"]
        s["x"] = normal(M, G * D, scale=2.0) + normal(1, G * D)
        s["w"] = 1.0 + uniform(-0.2, 0.2, G * D)
        s["b"] = uniform(-0.2, 0.2, G * D)
        s["z"] = normal(M, G * D) if case["gate"] else None
        if case["train"]:
            s["dy"] = normal(M, G * D)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = normal(M, K)
        s["W"] = normal(N, K, scale=1.0 / math.sqrt(K))
        s["bias"] = normal(N, scale=0.2)
        s["res"] = normal(M, N) if case["res"] else None
        if case["train"]:
            s["dy"] = normal(M, N)
    return s


# ----------------------------------------------------------------------------- the plain forms
def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _silu(x):
    return x * _sigmoid(x)


def _d_silu(x):
    s = _sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


def _gelu(x):
    return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))


def _d_gelu(x):
    return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)


ACTS = {"none": (lambda x: x, torch.ones_like), "silu": (_silu, _d_silu), "gelu": (_gelu, _d_gelu)}


def _f32(t):
    return None if t is None else t.float()


def _valid(s):
    """[B, T] truth values: whether a step lies inside its row."""
    c = s["case"]
    steps = torch.arange(c["T"], device="cuda")
    return torch.ones(c["B"], c["T"], dtype=torch.bool, device="cuda") if s["lens"] is None else steps < s["lens"][:, None]


def _plain_conv(s):
    c = s["case"]
    B, T, C, W = c["B"], c["T"], c["C"], c["W"]
    dt = DTYPES[c["dtype"]]
    ok = _valid(s)[:, :, None]
    x = torch.where(ok, s["x"].float(), 0.0)
    s0 = torch.zeros(B, W - 1, C, device="cuda") if s["s0"] is None else s["s0"].float()
    rows = torch.cat([s0, x], 1)                                   # [B, W - 1 + T, C]
    taps = rows.unfold(1, W, 1)                                    # [B, T, C, W], a view
    pre = (taps * s["w"]).sum(-1) + s["bias"]
    y = torch.where(ok, _silu(pre), 0.0).to(dt)
    last = torch.full((B,), T, device="cuda", dtype=torch.int64) if s["lens"] is None else s["lens"].long()
    at = last[:, None] + torch.arange(W - 1, device="cuda")
    s_T = torch.gather(rows, 1, at[:, :, None].expand(B, W - 1, C)).to(dt)
    if not c["train"]:
        return y, s_T
    dpre = torch.where(ok, s["dy"].float() * _d_silu(pre), 0.0)
    dw = (taps * dpre[..., None]).sum((0, 1))
    dbias = dpre.sum((0, 1))
    wide = torch.nn.functional.pad(dpre, (0, 0, W - 1, W - 1))     # [B, T + 2 (W - 1), C]
    drows = (wide.unfold(1, W, 1) * s["w"].flip(1)).sum(-1)        # [B, T + W - 1, C]
    dx = torch.where(ok, drows[:, W - 1:], 0.0).to(dt)
    ds0 = drows[:, :W - 1].to(dt) if s["s0"] is not None else None
    return {"y": y, "s_T": s_T, "dx": dx, "dw": dw, "dbias": dbias, "ds0": ds0}


def _recur(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dimension 1 (h[-1] = 0), by doubling."""
    step, T = 1, a.shape[1]
    while step < T:
        b = torch.cat([b[:, :step], torch.addcmul(b[:, step:], a[:, step:], b[:, :-step])], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _plain_scan(s):
    c = s["case"]
    B, T, C, N, G = c["B"], c["T"], c["C"], c["N"], c["G"]
    dt = DTYPES[c["dtype"]]
    ok = _valid(s)[:, :, None]
    u, z = torch.where(ok, s["u"].float(), 0.0), s["z"].float()
    Bc = s["B"].float().repeat_interleave(C // G, 2)               # [B, T, C, N]
    Cc = s["C"].float().repeat_interleave(C // G, 2)
    raw = s["dt"].float() + s["dt_bias"]
    step = torch.where(ok, torch.clamp(raw, min=0.0) + torch.log1p(torch.exp(-torch.abs(raw))), 0.0)
    A = -torch.exp(s["A_log"])
    a = torch.exp(step[..., None] * A)
    b = (step * u)[..., None] * Bc
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    h = _recur(a, b)
    h_T = h[:, -1].clone()
    core = (h * Cc).sum(-1) + s["D"] * u
    y = torch.where(ok, core * _silu(z), 0.0).to(dt)
    if not c["train"]:
        return y, h_T
    dy = torch.where(ok, s["dy"].float(), 0.0)
    dcore = dy * _silu(z)
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)   # the decay that follows each step
    e = _recur(later.flip(1), (dcore[..., None] * Cc).flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None], h[:, :-1]], 1)
    kept = e * a * before
    dsu = (e * Bc).sum(-1)
    dstep = (kept * A).sum(-1) + dsu * u
    ddt = torch.where(ok, dstep * _sigmoid(raw), 0.0)
    return {
        "y": y, "h_T": h_T,
        "du": (dsu * step + s["D"] * dcore).to(dt), "ddt": ddt.to(dt),
        "dA_log": (kept * step[..., None]).sum((0, 1)) * A,
        "dB": ((step * u)[..., None] * e).view(B, T, G, C // G, N).sum(3).to(dt),
        "dC": (dcore[..., None] * h).view(B, T, G, C // G, N).sum(3).to(dt),
        "dD": (dcore * u).sum((0, 1)), "ddt_bias": ddt.sum((0, 1)),
        "dz": torch.where(ok, dy * core * _d_silu(z), 0.0).to(dt),
        "dh0": a[:, 0] * e[:, 0] if s["h0"] is not None else None,
    }


def _plain_norm(s):
    c = s["case"]
    M, G, D = c["M"], c["G"], c["D"]
    dt = DTYPES[c["dtype"]]
    x = s["x"].float().view(M, G, D)
    w, b = s["w"].view(G, D), s["b"].view(G, D)
    off = x - x.mean(-1, keepdim=True)
    inv = 1.0 / torch.sqrt((off * off).mean(-1, keepdim=True) + EPS)
    xh = off * inv
    aff = xh * w + b
    z = None if s["z"] is None else s["z"].float().view(M, G, D)
    y = (_silu(aff) if z is None else aff * _silu(z)).view(M, G * D).to(dt)
    if not c["train"]:
        return y
    dy = s["dy"].float().view(M, G, D)
    daff = dy * (_d_silu(aff) if z is None else _silu(z))
    dxh = daff * w
    dx = inv * (dxh - dxh.mean(-1, keepdim=True) - xh * (dxh * xh).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.view(M, G * D).to(dt), "dw": (daff * xh).sum(0).view(G * D), "db": daff.sum(0).view(G * D),
            "dz": None if z is None else (dy * aff * _d_silu(z)).view(M, G * D).to(dt)}


def _plain_linear(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    act, d_act = ACTS[c["act"]]
    x, W = s["x"].float(), s["W"].float()
    pre = x @ W.t() + s["bias"].float()
    y = act(pre)
    if s["res"] is not None:
        y = y + s["res"].float()
    if not c["train"]:
        return y.to(dt)
    dpre = s["dy"].float() * d_act(pre)
    return {"y": y.to(dt), "dx": (dpre @ W).to(dt), "dW": (dpre.t() @ x).to(dt), "dbias": dpre.sum(0).to(dt)}


PLAIN = {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm, "linear": _plain_linear}


# ------------------------------------------------------------------------- the library's calls
def _own_conv(s):
    import gated_delta_rule_22_gb300 as gdn
    y, s_T = gdn.gdn_conv_fwd(s["x"], s["w"], s["bias"], s["s0"], s["lens"], act="silu")
    if not s["case"]["train"]:
        return y, s_T
    d = gdn.gdn_conv_bwd(s["x"], s["w"], s["dy"], s["bias"], s["s0"], s["lens"], act="silu", want_ds0=s["s0"] is not None)
    return {"y": y, "s_T": s_T, "dx": d["dx"], "dw": d["dw"], "dbias": d["dbias"], "ds0": d["ds0"]}


def _own_scan(s):
    import gated_delta_rule_22_gb300 as gdn
    train = s["case"]["train"]
    y, h_T, ckpt = gdn.gdn_scan_fwd(s["u"], s["dt"], s["A_log"], s["B"], s["C"], s["D"], s["dt_bias"], s["z"], s["h0"],
                                    s["lens"], want_ckpt=train)
    if not train:
        return y, h_T
    d = gdn.gdn_scan_bwd(s["u"], s["dt"], s["A_log"], s["B"], s["C"], ckpt, s["dy"], s["D"], s["dt_bias"], s["z"],
                         s["lens"], want_dh0=s["h0"] is not None)
    return {"y": y, "h_T": h_T, **{n: d[n] for n in ("du", "ddt", "dA_log", "dB", "dC", "dD", "ddt_bias", "dz", "dh0")}}


def _own_norm(s):
    import gated_delta_rule_22_gb300 as gdn
    c = s["case"]
    y, stats = gdn.gdn_norm_fwd(s["x"], c["G"], s["w"], s["b"], s["z"], act="silu", eps=EPS, want_stats=c["train"])
    if not c["train"]:
        return y
    d = gdn.gdn_norm_bwd(s["x"], c["G"], stats, s["dy"], s["w"], s["b"], s["z"], act="silu")
    return {"y": y, "dx": d["dx"], "dw": d["dw"], "db": d["db"], "dz": d["dz"]}


def _own_linear(s):
    import gated_delta_rule_22_gb300 as gdn
    c = s["case"]
    y, pre = gdn.gdn_linear_fwd(s["x"], s["W"], s["bias"], s["res"], act=c["act"], want_pre=c["train"] and c["act"] != "none")
    if not c["train"]:
        return y
    d = gdn.gdn_linear_bwd(s["x"], s["W"], s["dy"], pre, act=c["act"])
    return {"y": y, "dx": d["dx"], "dW": d["dW"], "dbias": d["dbias"]}


OWN = {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm, "linear": _own_linear}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "conv":
        n, W = case["B"] * case["T"] * case["C"], case["W"]
        state = case["B"] * (W - 1) * case["C"] * e * (2 if case["state"] else 1)
        fwd = 2 * n * e + case["C"] * (W + 1) * 4 + state
        if not case["train"]:
            return {"bytes": fwd, "flops": n * (2 * W + 4)}
        return {"bytes": fwd + 2 * n * e + case["C"] * (W + 1) * 4, "flops": n * (2 * W + 4) + n * (6 * W + 10)}
    if case["op"] == "scan":
        n, N = case["B"] * case["T"] * case["C"], case["N"]
        small = 2 * case["B"] * case["T"] * case["G"] * N * e
        state = case["B"] * case["C"] * N * 4
        fwd = 4 * n * e + small + case["C"] * (N + 2) * 4 + state * (2 if case["state"] else 1)
        if not case["train"]:
            return {"bytes": fwd, "flops": n * (6 * N + 10)}
        return {"bytes": fwd + 4 * n * e + small + case["C"] * (N + 2) * 4, "flops": n * (6 * N + 10) + n * (16 * N + 20)}
    if case["op"] == "norm":
        n, C = case["M"] * case["G"] * case["D"], case["G"] * case["D"]
        read = 2 if case["gate"] else 1
        fwd = (read + 1) * n * e + 2 * C * 4
        if not case["train"]:
            return {"bytes": fwd, "flops": 12 * n}
        return {"bytes": fwd + (read + 1) * n * e + 2 * C * 4, "flops": 36 * n}
    M, N, K = case["M"], case["N"], case["K"]
    fwd = (M * K + N * K + N + M * N * (2 if case["res"] else 1)) * e
    if not case["train"]:
        return {"bytes": fwd, "flops": 2 * M * N * K}
    return {"bytes": fwd + (M * N + M * K + N * K + N) * e, "flops": 6 * M * N * K}


# --------------------------------------------------------------- the definitions, in 64 bits
def _f64(t):
    return None if t is None else t.double()


def _sig64(x):
    return torch.special.expit(x)


def _exact_conv(s):
    c = s["case"]
    B, T, C, W = c["B"], c["T"], c["C"], c["W"]
    x, w, bias, s0 = _f64(s["x"]), _f64(s["w"]), _f64(s["bias"]), _f64(s["s0"])
    lens = [T] * B if s["lens"] is None else s["lens"].tolist()
    y, s_T = torch.zeros_like(x), torch.zeros(B, W - 1, C, dtype=torch.float64, device="cuda")
    out = {"y": y, "s_T": s_T}
    if c["train"]:
        dy = _f64(s["dy"])
        out.update(dx=torch.zeros_like(x), dw=torch.zeros(C, W, dtype=torch.float64, device="cuda"),
                   dbias=torch.zeros(C, dtype=torch.float64, device="cuda"), ds0=None if s0 is None else torch.zeros_like(s0))
    for b in range(B):
        L = lens[b]
        head = torch.zeros(W - 1, C, dtype=torch.float64, device="cuda") if s0 is None else s0[b]
        rows = torch.cat([head, x[b, :L]])
        s_T[b] = rows[L:L + W - 1]
        if L == 0:
            if c["train"] and s0 is not None:
                out["ds0"][b] = 0.0
            continue
        pre = bias.expand(L, C).clone()
        for j in range(W):
            pre += w[:, j] * rows[j:j + L]
        sg = _sig64(pre)
        y[b, :L] = pre * sg
        if c["train"]:
            dpre = dy[b, :L] * sg * (1 + pre * (1 - sg))
            drows = torch.zeros_like(rows)
            for j in range(W):
                drows[j:j + L] += w[:, j] * dpre
                out["dw"][:, j] += (rows[j:j + L] * dpre).sum(0)
            out["dbias"] += dpre.sum(0)
            out["dx"][b, :L] = drows[W - 1:]
            if s0 is not None:
                out["ds0"][b] = drows[:W - 1]
    return out if c["train"] else (y, s_T)


def _exact_scan(s):
    c = s["case"]
    B, T, C, N, G = c["B"], c["T"], c["C"], c["N"], c["G"]
    per = C // G
    u, z, raw = _f64(s["u"]), _f64(s["z"]), _f64(s["dt"]) + _f64(s["dt_bias"])
    Bm, Cm, D, A = _f64(s["B"]), _f64(s["C"]), _f64(s["D"]), -torch.exp(_f64(s["A_log"]))
    lens = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"]
    h = torch.zeros(B, C, N, dtype=torch.float64, device="cuda") if s["h0"] is None else _f64(s["h0"])
    d = torch.where(raw > 30, raw, torch.log1p(torch.exp(torch.clamp(raw, max=30.0))))
    wide = lambda m, t: m[:, t, :, None, :].expand(B, G, per, N).reshape(B, C, N)  # noqa: E731
    y = torch.zeros_like(u)
    hs = [h]
    gate = z * _sig64(z)
    core = torch.zeros_like(u)
    for t in range(T):
        on = (t < lens)[:, None, None]
        new = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * u[:, t])[:, :, None] * wide(Bm, t)
        h = torch.where(on, new, h)
        core[:, t] = (h * wide(Cm, t)).sum(2) + D * u[:, t]
        y[:, t] = torch.where(on[:, :, 0], core[:, t] * gate[:, t], 0.0)
        if c["train"]:
            hs.append(h)
    if not c["train"]:
        return y, h
    dy = _f64(s["dy"])
    out = {"y": y, "h_T": h}
    for n, like in (("du", u), ("ddt", u), ("dB", Bm), ("dC", Cm), ("dz", u)):
        out[n] = torch.zeros_like(like)
    dA, dD = torch.zeros_like(A), torch.zeros_like(D)
    e = torch.zeros_like(h)
    sg = _sig64(z)
    for t in range(T - 1, -1, -1):
        on2 = (t < lens)[:, None]
        on = on2[:, :, None]
        dc = torch.where(on2, dy[:, t] * gate[:, t], 0.0)
        out["dz"][:, t] = torch.where(on2, dy[:, t] * core[:, t] * sg[:, t] * (1 + z[:, t] * (1 - sg[:, t])), 0.0)
        e = e + dc[:, :, None] * wide(Cm, t)
        out["dC"][:, t] = (dc[:, :, None] * hs[t + 1]).view(B, G, per, N).sum(2)
        a = torch.exp(d[:, t, :, None] * A)
        through = torch.where(on, e * a * hs[t], 0.0)
        dsu = torch.where(on2, (e * wide(Bm, t)).sum(2), 0.0)
        out["dB"][:, t] = torch.where(on, e * (d[:, t] * u[:, t])[:, :, None], 0.0).view(B, G, per, N).sum(2)
        out["ddt"][:, t] = ((through * A).sum(2) + dsu * u[:, t]) * _sig64(raw[:, t])
        out["du"][:, t] = dsu * d[:, t] + D * dc
        dA += (through * d[:, t, :, None]).sum(0)
        dD += (dc * u[:, t]).sum(0)
        e = torch.where(on, e * a, e)
    out.update(dA_log=dA * A, dD=dD, ddt_bias=out["ddt"].sum((0, 1)), dh0=e if s["h0"] is not None else None)
    return out


def _exact_norm(s):
    c = s["case"]
    M, G, D = c["M"], c["G"], c["D"]
    x, w, b, z = _f64(s["x"]).view(M, G, D), _f64(s["w"]).view(G, D), _f64(s["b"]).view(G, D), _f64(s["z"])
    var, mean = torch.var_mean(x, 2, correction=0, keepdim=True)
    sd = torch.sqrt(var + EPS)
    xh = (x - mean) / sd
    aff = xh * w + b
    act = aff if z is None else z.view(M, G, D)
    sg = _sig64(act)
    y = aff * sg if z is None else aff * act * sg
    if not c["train"]:
        return y.view(M, G * D)
    dy = _f64(s["dy"]).view(M, G, D)
    slope = sg * (1 + act * (1 - sg))
    daff = dy * slope if z is None else dy * act * sg
    g = daff * w
    dx = (g - g.mean(2, keepdim=True) - xh * (g * xh).mean(2, keepdim=True)) / sd
    return {"y": y.view(M, G * D), "dx": dx.view(M, G * D), "dw": torch.einsum("mgd,mgd->gd", daff, xh).reshape(-1),
            "db": daff.sum(0).reshape(-1), "dz": None if z is None else (dy * aff * slope).view(M, G * D)}


def _exact_linear(s):
    c = s["case"]
    x, W, bias, res = _f64(s["x"]), _f64(s["W"]), _f64(s["bias"]), _f64(s["res"])
    pre = torch.addmm(bias, x, W.t())
    if c["act"] == "silu":
        sg = _sig64(pre)
        y, slope = pre * sg, sg * (1 + pre * (1 - sg))
    elif c["act"] == "gelu":
        cdf = torch.special.ndtr(pre)
        y, slope = pre * cdf, cdf + pre * torch.exp(-pre * pre / 2) / math.sqrt(2 * math.pi)
    else:
        y, slope = pre, torch.ones_like(pre)
    y = y if res is None else y + res
    if not c["train"]:
        return y
    dpre = _f64(s["dy"]) * slope
    return {"y": y, "dx": dpre @ W, "dW": dpre.t() @ x, "dbias": dpre.sum(0)}


EXACT = {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm, "linear": _exact_linear}


def exact(case, seed):
    if case["op"] == "scan" and case["train"] and case["B"] * case["T"] * case["C"] * case["N"] > 3e8:
        return None  # the states of every step in 64 bits do not fit beside the rest
    return EXACT[case["op"]](prepare(case, seed))

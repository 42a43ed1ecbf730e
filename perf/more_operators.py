"""Linear attention with a decay for each head, and the norms around a block, as measured cases.

A block of a recurrent model runs a norm, a mixer and an addition onto the residual stream. The mixers of
the library are the gated delta rule and the selective scan; the one measured here is linear attention
whose state decays by a constant of each head (chunked for prompts and training, recurrent for single
tokens). Around every mixer stand a norm of the block's output, its gate and residual scale, the addition,
and the norm in front of the next block: one operator, measured here too.

`own = False` computes each operator in its plain form: elementary torch operations in 32 bits (powers of
the decay from 64), rounded once at the end. `own = True` calls the library.

    linattn  S_t = g S_{t-1} + v_t k_t^T,  y_t = S_t q_t,  a constant g of each value head; value head h
             reads key head h // (Hv / Hk)
    resnorm  n = h / rms(h) w_post,  r = x + scale act(z) n,  y = r / rms(r) w_pre;  rms(a) =
             sqrt(mean(a^2) + eps);  z has one row for each row of x, or one for each sequence
"""
import math

import torch

own = False

EPS = 1e-5
CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One generated token for a single user: two launches' latency is all there is.
        dict(name="linattn-token-one", op="linattn", dtype="bf16", B=1, T=1, Hk=16, Hv=32, Dk=128, Dv=128, state=True, ragged=False, train=False),
        # One generated token for each of 64 sequences: the state is read and written once.
        dict(name="linattn-token", op="linattn", dtype="bf16", B=64, T=1, Hk=16, Hv=32, Dk=128, Dv=128, state=True, ragged=False, train=False),
        # Four prompts of different lengths, padded to the longest, that continue a cached prefix.
        dict(name="linattn-prompt", op="linattn", dtype="bf16", B=4, T=2048, Hk=16, Hv=32, Dk=128, Dv=128, state=True, ragged=True, train=False),
        # One GPU's share of a long-context layer (2 of 16 key heads, 8 of 64 value heads): few heads, a long sequence.
        dict(name="linattn-long", op="linattn", dtype="bf16", B=1, T=32768, Hk=2, Hv=8, Dk=192, Dv=128, state=False, ragged=False, train=False),
        # A training step, forward and backward: every value head with keys of its own.
        dict(name="linattn-train", op="linattn", dtype="bf16", B=4, T=4096, Hk=32, Hv=32, Dk=128, Dv=128, state=False, ragged=False, train=True),
        # Training in 32 bits on short ragged rows, odd sizes, shared keys, a carried state.
        dict(name="linattn-train-odd", op="linattn", dtype="f32", B=3, T=333, Hk=3, Hv=6, Dk=40, Dv=75, state=True, ragged=True, train=True),
        # The residual stream of 64 generated tokens between two blocks.
        dict(name="resnorm-token", op="resnorm", dtype="bf16", B=64, T=1, D=2048, post=True, gate="none", act="none", scale=True, train=False),
        # Prompts whose block's output is gated by one row for each sequence (a condition's modulation).
        dict(name="resnorm-prompt", op="resnorm", dtype="bf16", B=4, T=2048, D=4096, post=True, gate="sequence", act="none", scale=False, train=False),
        # A training step's share of the batched layer: forward and backward over 8 x 4096 steps.
        dict(name="resnorm-train", op="resnorm", dtype="bf16", B=8, T=4096, D=2048, post=True, gate="none", act="none", scale=True, train=True),
        # Training in 32 bits, odd sizes, a gate with an activation for every step, no norm behind the block.
        dict(name="resnorm-train-odd", op="resnorm", dtype="f32", B=3, T=333, D=1030, post=False, gate="step", act="silu", scale=True, train=True),
    ]


def _log_size(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    use = rng.choice(["token", "prompt", "train"])
    train = use == "train"
    if rng.random() < 0.6:
        Hk, group = _log_size(rng, 1, 16), rng.choice([1, 1, 2, 3, 4])
        width = lambda: rng.choice([64, 128, 128, 192, 256, rng.randint(8, 256)])  # noqa: E731
        Dk, Dv = width(), width()
        T = 1 if use == "token" else _log_size(rng, 2, 16384)
        B = _log_size(rng, 1, 64) if use == "token" else rng.randint(1, 8)
        most = 4 * 4096 * 32 * 2 * 128 // (2 if dtype == "f32" else 1)
        while B * T * Hk * group * (Dk + Dv) > most:
            B, T = max(1, B // 2), max(2, T // 2)
        return dict(op="linattn", dtype=dtype, B=B, T=T, Hk=Hk, Hv=Hk * group, Dk=Dk, Dv=Dv, state=use == "token" or rng.random() < 0.5,
                    ragged=use != "token" and rng.random() < 0.4, train=train)
    D = _log_size(rng, 64, 8192)
    if rng.random() < 0.5:
        D = max(64, D // 64 * 64)
    T = 1 if use == "token" else _log_size(rng, 16, 4096)
    B = _log_size(rng, 1, 128) if use == "token" else rng.randint(1, 8)
    while B * T * D > 8 * 4096 * 2048 // (2 if dtype == "f32" else 1):
        T = max(1, T // 2)
    return dict(op="resnorm", dtype=dtype, B=B, T=T, D=D, post=rng.random() < 0.6, gate=rng.choice(["none", "sequence", "step"]),
                act=rng.choice(["none", "silu"]), scale=rng.random() < 0.5, train=train)


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    def uniform(low, high, *shape):
        return torch.rand(*shape, generator=gen, device="cuda") * (high - low) + low

    s = {"case": case}
    B, T = case["B"], case["T"]
    if case["op"] == "linattn":
        Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
        s["q"], s["k"], s["v"] = normal(B, T, Hk, Dk, scale=Dk ** -0.5), normal(B, T, Hk, Dk), normal(B, T, Hv, Dv)
        # the heads' memories spread from a step or two to some hundreds of steps
        s["g"] = torch.exp(-torch.exp2(-8.0 * (torch.arange(Hv, device="cuda") + uniform(0.0, 1.0, Hv)) / Hv))
        s["S0"] = normal(B, Hv, Dv, Dk, scale=2.0, dtype=torch.float32) if case["state"] else None
        s["lens"] = None
        if case["ragged"]:  # one row is full, one has no valid step at all, the rest lie between
            lens = torch.randint(1, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
            lens[0] = T
            if B > 2:
                lens[B - 1] = 0
            s["lens"] = lens
        if case["train"]:
            s["dy"] = normal(B, T, Hv, Dv)
            s["dS_T"] = normal(B, Hv, Dv, Dk, scale=0.1, dtype=torch.float32) if case["state"] else None
        return s
    D = case["D"]
    s["x"], s["h"] = normal(B, T, D, scale=2.0), normal(B, T, D, scale=0.7)
    s["z"] = None if case["gate"] == "none" else normal(B, D) if case["gate"] == "sequence" else normal(B, T, D)
    s["scale"] = uniform(0.2, 0.8, D) if case["scale"] else None
    s["w_post"] = 1.0 + uniform(-0.2, 0.2, D) if case["post"] else None
    s["w_pre"] = 1.0 + uniform(-0.2, 0.2, D)
    if case["train"]:
        s["dy"], s["dr"] = normal(B, T, D), normal(B, T, D)
    return s


# ----------------------------------------------------------------------------- the plain forms
def _powers(g, n):
    """g^n in 64 bits, rounded to 32: g [Hv, 1, ...], n whole numbers; 0 where n < 0."""
    return torch.where(n >= 0, torch.pow(g.double(), n.clamp(min=0).double()), 0.0).float()


def _chunks(x):
    """[B, T, H, D] -> [B, H, N, CHUNK, D], zeros behind the last step."""
    B, T, H, D = x.shape
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -T % CHUNK))
    return x.view(B, -1, CHUNK, H, D).permute(0, 3, 1, 2, 4)


def _decayed(a, b, c, g):
    """y_t = sum_{s <= t} g^(t-s) (a_t . b_s) c_s, heads first in g: within chunks of steps, and through the
    chunks' sums of c b^T."""
    T, H = a.shape[1:3]
    a, b, c = _chunks(a), _chunks(b), _chunks(c)
    i = torch.arange(CHUNK, device="cuda")
    n = torch.arange(a.shape[2], device="cuda")
    g = g.view(H, 1, 1)
    inside = (a @ b.transpose(-1, -2)) * _powers(g, i[:, None] - i)[:, None]
    sums = (c * _powers(g, CHUNK - 1 - i[None, :, None])[:, None]).transpose(-1, -2) @ b            # [B, H, N, Dc, Db]
    before = _powers(g, (n[:, None] - n - 1) * CHUNK)                                                # [H, N, N]
    state = (before @ sums.flatten(-2)).view(sums.shape)
    y = inside @ c + (a @ state.transpose(-1, -2)) * _powers(g, i[None, :, None] + 1)[:, None]
    return y.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :T]


def _plain_linattn(s):
    c = s["case"]
    B, T, Hk, Hv, Dk, Dv = (c[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    dt = DTYPES[c["dtype"]]
    g = s["g"]
    q, k = (s[n].float().repeat_interleave(Hv // Hk, 2) for n in ("q", "k"))
    v = s["v"].float()
    if T == 1 and not c["train"]:
        S = g[:, None, None] * s["S0"] + v[:, 0, :, :, None] * k[:, 0, :, None, :]
        return (S * q[:, 0, :, None, :]).sum(-1)[:, None].to(dt), S
    steps = torch.arange(T, device="cuda")
    lens = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"]
    ok = (steps < lens[:, None])[:, :, None, None]
    q, k, v = (torch.where(ok, t, 0.0) for t in (q, k, v))
    past = _powers(g.view(1, 1, Hv, 1), steps[None, :, None, None] + 1)                              # g^(t+1)
    left = _powers(g.view(1, 1, Hv, 1), lens[:, None, None, None] - 1 - steps[None, :, None, None])  # g^(len-1-t)
    whole = _powers(g.view(1, Hv, 1, 1), lens[:, None, None, None])
    y = _decayed(q, k, v, g)
    S_T = (v * left).permute(0, 2, 3, 1) @ k.transpose(1, 2)
    if s["S0"] is not None:
        y = y + past * (q.transpose(1, 2) @ s["S0"].transpose(-1, -2)).transpose(1, 2)
        S_T = S_T + whole * s["S0"]
    y = torch.where(ok, y, 0.0).to(dt)
    if not c["train"]:
        return y, S_T
    dy = torch.where(ok, s["dy"].float(), 0.0)
    back = lambda a, b, e: _decayed(a.flip(1), b.flip(1), e.flip(1), g).flip(1)  # noqa: E731
    dq, dk, dv = _decayed(dy, v, k, g), back(v, dy, q), back(k, q, dy)
    dS0 = (dy * past).permute(0, 2, 3, 1) @ q.transpose(1, 2)
    if s["S0"] is not None:
        dq = dq + past * (dy.transpose(1, 2) @ s["S0"]).transpose(1, 2)
        dk = dk + left * (v.transpose(1, 2) @ s["dS_T"]).transpose(1, 2)
        dv = dv + left * (k.transpose(1, 2) @ s["dS_T"].transpose(-1, -2)).transpose(1, 2)
        dS0 = dS0 + whole * s["dS_T"]
    dq, dk = (torch.where(ok, t, 0.0).view(B, T, Hk, Hv // Hk, Dk).sum(3).to(dt) for t in (dq, dk))
    return {"y": y, "S_T": S_T, "dq": dq, "dk": dk, "dv": torch.where(ok, dv, 0.0).to(dt), "dS0": dS0 if c["state"] else None}


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _plain_resnorm(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    x, h = s["x"].float(), s["h"].float()
    rms = lambda t: torch.sqrt((t * t).mean(-1, keepdim=True) + EPS)  # noqa: E731
    one = torch.ones(c["D"], device="cuda")
    scale = one if s["scale"] is None else s["scale"]
    z = None if s["z"] is None else s["z"].float()[:, None] if c["gate"] == "sequence" else s["z"].float()
    gate = one if z is None else z * _sigmoid(z) if c["act"] == "silu" else z
    in_h = rms(h) if c["post"] else None
    hh = h / in_h if c["post"] else h
    n = hh * s["w_post"] if c["post"] else hh
    r = x + scale * gate * n
    in_r = rms(r)
    rh = r / in_r
    y = rh * s["w_pre"]
    if not c["train"]:
        return r.to(dt), y.to(dt)
    dy = s["dy"].float()
    e = dy * s["w_pre"]
    dr = s["dr"].float() + (e - rh * (e * rh).mean(-1, keepdim=True)) / in_r
    dn = dr * scale * gate
    dh = dn
    if c["post"]:
        e = dn * s["w_post"]
        dh = (e - hh * (e * hh).mean(-1, keepdim=True)) / in_h
    out = {"r": r.to(dt), "y": y.to(dt), "dx": dr.to(dt), "dh": dh.to(dt), "dw_pre": (dy * rh).sum((0, 1)),
           "dw_post": (dn * hh).sum((0, 1)) if c["post"] else None, "dscale": None, "dz": None}
    if s["scale"] is not None:
        out["dscale"] = (dr * gate * n).sum((0, 1))
    if z is not None:
        slope = _sigmoid(z) * (1.0 + z * (1.0 - _sigmoid(z))) if c["act"] == "silu" else 1.0
        dz = dr * scale * n * slope
        out["dz"] = (dz.sum(1) if c["gate"] == "sequence" else dz).to(dt)
    return out


PLAIN = {"linattn": _plain_linattn, "resnorm": _plain_resnorm}


# ------------------------------------------------------------------------- the library's calls
def _own_linattn(s):
    import gated_delta_rule_22_gb300 as gdn
    y, S_T = gdn.gdn_linattn_fwd(s["q"], s["k"], s["v"], s["g"], s["S0"], s["lens"])
    if not s["case"]["train"]:
        return y, S_T
    d = gdn.gdn_linattn_bwd(s["q"], s["k"], s["v"], s["g"], s["dy"], s["S0"], s["lens"], s["dS_T"], want_dS0=s["case"]["state"])
    return {"y": y, "S_T": S_T, "dq": d["dq"], "dk": d["dk"], "dv": d["dv"], "dS0": d["dS0"]}


def _own_resnorm(s):
    import gated_delta_rule_22_gb300 as gdn
    c = s["case"]
    form = dict(post=c["post"], act=c["act"], eps=EPS)
    r, y, stats = gdn.gdn_resnorm_fwd(s["x"], s["h"], s["z"], s["scale"], s["w_post"], s["w_pre"], want_stats=c["train"], **form)
    if not c["train"]:
        return r, y
    d = gdn.gdn_resnorm_bwd(s["x"], s["h"], stats, s["dy"], s["dr"], s["z"], s["scale"], s["w_post"], s["w_pre"], **form)
    return {"r": r, "y": y, **{n: d[n] for n in ("dx", "dh", "dw_pre", "dw_post", "dscale", "dz")}}


OWN = {"linattn": _own_linattn, "resnorm": _own_resnorm}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linattn":
        steps, Hk, Hv, Dk, Dv = case["B"] * case["T"], case["Hk"], case["Hv"], case["Dk"], case["Dv"]
        keys, values, state = steps * Hk * Dk * e, steps * Hv * Dv * e, case["B"] * Hv * Dv * Dk * 4
        # forward: q, k, v in, y out, the state out (and in); a step adds one product to the state and takes one from it
        bytes_, flops = 2 * keys + 2 * values + state * (2 if case["state"] else 1) + Hv * 4, 4 * steps * Hv * Dk * Dv
        if case["train"]:  # backward: q, k, v, dy in, dq, dk, dv out; the state, its adjoint, and three products with them
            bytes_ += 4 * keys + 3 * values + (3 * state if case["state"] else 0)
            flops += 10 * steps * Hv * Dk * Dv
        return {"bytes": bytes_, "flops": flops}
    n, D = case["B"] * case["T"] * case["D"], case["D"]
    gate = 0 if case["gate"] == "none" else n * e if case["gate"] == "step" else case["B"] * D * e
    weights = (1 + int(case["post"]) + int(case["scale"])) * D * 4
    if not case["train"]:
        return {"bytes": 4 * n * e + gate + weights, "flops": 12 * n}
    return {"bytes": 4 * n * e + gate + weights + 6 * n * e + 2 * gate + 2 * weights, "flops": 40 * n}


# --------------------------------------------------------------- the definitions, in 64 bits
def _exact_linattn(s):
    """The recurrence, step by step, and its adjoint, backwards."""
    c = s["case"]
    B, T, Hk, Hv, Dk, Dv = (c[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    own_key = torch.arange(Hv, device="cuda") // (Hv // Hk)
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    g = s["g"].double()[:, None, None]
    lens = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"]
    S = torch.zeros(B, Hv, Dv, Dk, dtype=torch.float64, device="cuda") if s["S0"] is None else s["S0"].double()
    y = torch.zeros_like(v)
    train = c["train"]
    dy = s["dy"].double() if train else None
    dq, dk, dv = (torch.zeros_like(t) for t in (q, k, v)) if train else (None, None, None)
    for t in range(T):
        on = (t < lens)[:, None, None]
        S = torch.where(on[..., None], g * S + v[:, t, :, :, None] * k[:, t, own_key][:, :, None], S)
        y[:, t] = torch.where(on, (S @ q[:, t, own_key][..., None])[..., 0], 0.0)
        if train:
            per_head = torch.where(on, (dy[:, t, :, None] @ S)[:, :, 0], 0.0)
            dq[:, t].index_add_(1, own_key, per_head)
    if not train:
        return y, S
    R = torch.zeros_like(S) if s["dS_T"] is None else s["dS_T"].double()
    for t in range(T - 1, -1, -1):
        on = (t < lens)[:, None, None]
        at = R + dy[:, t, :, :, None] * q[:, t, own_key][:, :, None]
        dk[:, t].index_add_(1, own_key, torch.where(on, (v[:, t, :, None] @ at)[:, :, 0], 0.0))
        dv[:, t] = torch.where(on, (at @ k[:, t, own_key][..., None])[..., 0], 0.0)
        R = torch.where(on[..., None], g * at, R)
    return {"y": y, "S_T": S, "dq": dq, "dk": dk, "dv": dv, "dS0": R if c["state"] else None}


def _exact_resnorm(s):
    """The formulas as one function of the inputs, and its gradients by reverse differentiation in 64 bits."""
    c = s["case"]
    names = [n for n in ("x", "h", "z", "scale", "w_post", "w_pre") if s[n] is not None]
    leaf = {n: s[n].double().requires_grad_(c["train"]) for n in names}
    h = leaf["h"]
    if c["post"]:
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * leaf["w_post"]
    if "z" in leaf:
        z = torch.nn.functional.silu(leaf["z"]) if c["act"] == "silu" else leaf["z"]
        h = h * (z.unsqueeze(1) if c["gate"] == "sequence" else z)
    if "scale" in leaf:
        h = h * leaf["scale"]
    r = leaf["x"] + h
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * leaf["w_pre"]
    if not c["train"]:
        return r, y
    grads = dict(zip(names, torch.autograd.grad([r, y], [leaf[n] for n in names], [s["dr"].double(), s["dy"].double()])))
    return {"r": r.detach(), "y": y.detach(), "dx": grads["x"], "dh": grads["h"], "dw_pre": grads["w_pre"], "dw_post": grads.get("w_post"),
            "dscale": grads.get("scale"), "dz": grads.get("z")}


EXACT = {"linattn": _exact_linattn, "resnorm": _exact_resnorm}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))

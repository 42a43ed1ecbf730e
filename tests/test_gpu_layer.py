"""GPU parity of the layer operators (through the C ABI's binding) against their float64
definitions, at the sizes, lengths, strides and masks where the kernels change their path.

Tolerances, relative 2-norm per output, fixed from the formats before the first run: float32
outputs 1e-5 (sums of up to some thousand float32 terms, each with a few ulp from the hardware's
exp2); bf16 outputs 5e-3 (one rounding gives up to 2^-9 of each element, 1.7e-3 of the norm; the
projection's backward rounds the pre-activation, dpre and the result, three such roundings)."""
import pytest

import gpu_harness as H

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layer_reference as R  # noqa: E402

TOL = {torch.float32: H.TOL["f32"], torch.bfloat16: H.TOL["bf16"]}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import os
    from gated_delta_rule_22_gb300 import binding
    if not os.path.exists(binding.LIB_PATH):
        from gated_delta_rule_22_gb300 import build
        build.build()
    import gated_delta_rule_22_gb300 as g
    return g


class Draw:
    def __init__(self, seed, dtype):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.dtype = TYPES[dtype]

    def normal(self, *shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, generator=self.g, device="cuda") * scale).to(dtype or self.dtype)

    def wide(self, B, T, C, pad, at, scale=1.0):
        """A [B, T, C] slice of a wider tensor (packed with pad = 0); what lies beside it is NaN."""
        if pad == 0:
            return self.normal(B, T, C, scale=scale)
        t = torch.full((B, T, C + pad), float("nan"), device="cuda", dtype=self.dtype)
        t[..., at:at + C] = self.normal(B, T, C, scale=scale)
        return t[..., at:at + C]


def poison(t, lens):
    """NaN and infinities in the steps behind each row's length."""
    if lens is not None and t is not None:
        for b, n in enumerate(lens.tolist()):
            t[b, max(n, 0):] = float("nan")
            t[b, max(n, 0)::2] = float("inf")
    return t


def clean(t, lens):
    if lens is None or t is None:
        return t
    t = t.clone()
    for b, n in enumerate(lens.tolist()):
        t[b, max(n, 0):] = 0.0
    return t


def d64(t):
    return None if t is None else t.detach().double()


def check(label, got, ref):
    bad = {}
    for n, r in ref.items():
        e = R.rel(got[n], r)
        if not e <= TOL[got[n].dtype]:
            bad[n] = e
    assert not bad, (label, bad)


# ---------------------------------------------------------------------------- convolution
CONV = [
    # B, T, C, W, dtype, pad, at, state, lens, act
    (2, 1, 64, 4, "bf16", 0, 0, True, None, "silu"),
    (3, 1, 37, 4, "f32", 0, 0, True, [1, 0, 1], "silu"),
    (1, 2, 8, 4, "f32", 0, 0, True, None, "silu"),
    (2, 3, 16, 4, "bf16", 8, 8, False, [2, 3], "silu"),
    (3, 130, 264, 4, "bf16", 0, 0, True, [130, 0, 7], "silu"),
    (2, 257, 33, 3, "bf16", 3, 1, True, [256, 300], "silu"),
    (1, 1000, 20, 2, "f32", 4, 4, False, None, "silu"),
    (2, 65, 12, 1, "f32", 0, 0, False, [64, -5], "silu"),
    (4, 513, 136, 4, "bf16", 8, 0, True, [1, 2, 3, 513], "none"),
    (2, 300, 1030, 4, "f32", 2, 2, True, None, "none"),
]


def conv_inputs(case):
    B, T, C, W, dtype, pad, at, state, lens, act = case
    r = Draw(B * 1000 + T + C, dtype)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    t = dict(x=poison(r.wide(B, T, C, pad, at), n), w=r.normal(C, W, scale=W ** -0.5, dtype=torch.float32),
             bias=r.normal(C, dtype=torch.float32), s0=r.normal(B, W - 1, C) if state else None)
    return t, n, poison(r.normal(B, T, C), n), r.normal(B, W - 1, C), act


@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(gdn, case):
    t, lens, dy, ds_T, act = conv_inputs(case)
    y, s_T = gdn.gdn_conv_fwd(t["x"], t["w"], t["bias"], t["s0"], lens, act=act)
    d = gdn.gdn_conv_bwd(t["x"], t["w"], dy, t["bias"], t["s0"], lens, ds_T, act=act, want_ds0=t["s0"] is not None)
    leaves = {k: d64(clean(v, lens) if k == "x" else v) for k, v in t.items()}
    (y64, s64), g = R.with_grads(lambda x, w, bias, s0: R.conv(x, w, bias, s0, lens, act), leaves,
                                 (d64(clean(dy, lens)), d64(ds_T)))
    check("conv", {"y": y, "s_T": s_T}, {"y": y64, "s_T": s64})
    assert torch.equal(s_T.double(), s64)              # a copy of inputs, no arithmetic
    check("conv grads", d, {"d" + k: v for k, v in g.items()})


def test_conv_without_bias_and_state_outputs(gdn):
    r = Draw(5, "bf16")
    x, w, dy = r.normal(2, 40, 72), r.normal(72, 4, dtype=torch.float32), r.normal(2, 40, 72)
    y, s_T = gdn.gdn_conv_fwd(x, w, want_s_T=False)
    assert s_T is None
    d = gdn.gdn_conv_bwd(x, w, dy, want_ds0=False)
    (y64, _), g = R.with_grads(lambda x, w: R.conv(x, w, None, None, None, "silu"), {"x": d64(x), "w": d64(w)}, (d64(dy), None))
    check("conv", {"y": y, **d}, {"y": y64, "dx": g["x"], "dw": g["w"]})


def test_conv_token_by_token_continues_the_prompt(gdn):
    """A prompt, then single steps with the state updated in place: the bits of one long call."""
    r = Draw(6, "bf16")
    x, w, bias = r.normal(3, 20, 136), r.normal(136, 4, dtype=torch.float32), r.normal(136, dtype=torch.float32)
    whole, s_end = gdn.gdn_conv_fwd(x, w, bias)
    y, s = gdn.gdn_conv_fwd(x[:, :17].contiguous(), w, bias)
    ys = [y]
    for t in range(17, 20):
        y, s2 = gdn.gdn_conv_fwd(x[:, t:t + 1], w, bias, s, s_T=s)
        assert s2 is s
        ys.append(y)
    assert torch.equal(torch.cat(ys, 1), whole) and torch.equal(s, s_end)


# ---------------------------------------------------------------------------------- scan
SCAN = [
    # B, T, C, N, G, dtype, pad, state, lens, gate, D and dt_bias
    (2, 1, 64, 16, 1, "bf16", 0, True, None, True, True),
    (3, 1, 35, 5, 5, "f32", 0, True, [1, 0, 1], True, True),
    (1, 2, 8, 4, 1, "f32", 0, False, None, False, False),
    (2, 15, 70, 16, 1, "f32", 0, True, [15, 3], True, True),
    (2, 16, 64, 16, 2, "bf16", 8, True, None, True, True),
    (2, 17, 66, 1, 2, "f32", 0, True, [16, 17], True, False),
    (1, 100, 200, 16, 2, "bf16", 0, False, None, True, True),
    (3, 130, 48, 11, 3, "f32", 4, True, [130, 0, 31], True, True),
    (2, 75, 40, 32, 1, "f32", 0, True, [75, 70], True, True),
    (1, 50, 33, 23, 1, "bf16", 3, True, None, False, True),
    (2, 40, 24, 64, 1, "f32", 0, True, None, True, True),
    (1, 47, 20, 49, 2, "bf16", 0, True, [33], True, True),
    (1, 700, 72, 16, 1, "f32", 0, True, None, True, True),          # split into segments
    (2, 1030, 20, 8, 2, "f32", 0, True, [1030, 600], True, True),   # split, one row ends inside
    (2, 515, 16, 40, 1, "bf16", 8, False, [0, 514], True, True),    # split, wide states
]


def scan_inputs(case):
    B, T, C, N, G, dtype, pad, state, lens, gate, full = case
    r = Draw(B * 1000 + T + C + N, dtype)
    f32 = torch.float32
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    bc = lambda: poison(r.wide(B, T, G * N, pad, 0).unflatten(2, (G, N)), n)  # noqa: E731
    t = dict(u=poison(r.wide(B, T, C, pad, pad), n), dt=poison(r.wide(B, T, C, pad, 0, scale=0.7), n),
             A_log=r.normal(C, N, scale=0.7, dtype=f32), B=bc(), C=bc(), D=r.normal(C, dtype=f32) if full else None,
             dt_bias=r.normal(C, dtype=f32) - 1.5 if full else None, z=poison(r.wide(B, T, C, pad, pad), n) if gate else None,
             h0=r.normal(B, C, N, dtype=f32) if state else None)
    return t, n, poison(r.normal(B, T, C), n), r.normal(B, C, N, dtype=f32)


@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan(gdn, case):
    t, lens, dy, dh_T = scan_inputs(case)
    order = ("u", "dt", "A_log", "B", "C", "D", "dt_bias", "z")
    args = [t[k] for k in order]
    y, h_T, ckpt = gdn.gdn_scan_fwd(*args, t["h0"], lens, want_ckpt=True)
    y2, h2, none = gdn.gdn_scan_fwd(*args, t["h0"], lens)              # a single step: the streaming kernel
    d = gdn.gdn_scan_bwd(*args[:5], ckpt, dy, *args[5:], lens, dh_T, want_dh0=t["h0"] is not None)
    strided = ("u", "dt", "B", "C", "z")
    leaves = {k: d64(clean(v, lens) if k in strided else v) for k, v in t.items()}
    (y64, h64), g = R.with_grads(lambda **k: R.scan(lens=lens, **k), leaves, (d64(clean(dy, lens)), d64(dh_T)))
    assert none is None
    for yy, hh in ((y, h_T), (y2, h2)):
        check("scan", {"y": yy, "h_T": hh}, {"y": y64, "h_T": h64})
    check("scan grads", d, {"d" + k: v for k, v in g.items()})


def test_scan_rows_of_length_zero_pass_the_state(gdn):
    t, lens, dy, dh_T = scan_inputs((3, 130, 48, 11, 3, "f32", 4, True, [130, 0, 31], True, True))
    y, h_T, ckpt = gdn.gdn_scan_fwd(t["u"], t["dt"], t["A_log"], t["B"], t["C"], t["D"], t["dt_bias"], t["z"], t["h0"], lens,
                                    want_ckpt=True)
    assert torch.equal(h_T[1], t["h0"][1]) and not y[1].any() and not y[2, 31:].any()
    d = gdn.gdn_scan_bwd(t["u"], t["dt"], t["A_log"], t["B"], t["C"], ckpt, dy, t["D"], t["dt_bias"], t["z"], lens, dh_T)
    assert torch.equal(d["dh0"][1], dh_T[1])
    for k in ("du", "ddt", "dB", "dC", "dz"):
        assert not d[k][1].any() and not d[k][2, 31:].any(), k


def test_scan_gradient_against_differences(gdn):
    """The kernels' gradients against central differences of the float64 definition along random
    directions."""
    t, lens, dy, dh_T = scan_inputs((2, 40, 24, 64, 1, "f32", 0, True, None, True, True))
    args = [t[k] for k in ("u", "dt", "A_log", "B", "C", "D", "dt_bias", "z")]
    _, _, ckpt = gdn.gdn_scan_fwd(*args, t["h0"], want_ckpt=True)
    d = gdn.gdn_scan_bwd(*args[:5], ckpt, dy, *args[5:], None, dh_T)
    leaves = {k: d64(v) for k, v in t.items()}

    def loss(over):
        y, h = R.scan(lens=None, **{**leaves, **over})
        return ((y * d64(dy)).sum() + (h * d64(dh_T)).sum()).item()

    r = Draw(9, "f32")
    for k, v in leaves.items():
        way = r.normal(*v.shape).double()
        h = 1e-5
        numeric = (loss({k: v + h * way}) - loss({k: v - h * way})) / (2 * h)
        scale = torch.linalg.vector_norm(d["d" + k].double()).item() * torch.linalg.vector_norm(way).item()
        assert abs((d["d" + k].double() * way).sum().item() - numeric) <= 1e-5 * scale, k


def test_scan_token_by_token_continues_the_prompt(gdn):
    t, _, _, _ = scan_inputs((2, 40, 72, 16, 2, "f32", 0, True, None, True, True))
    cut = lambda a, b: [t["u"][:, a:b].contiguous(), t["dt"][:, a:b].contiguous(), t["A_log"], t["B"][:, a:b].contiguous(),  # noqa: E731
                        t["C"][:, a:b].contiguous(), t["D"], t["dt_bias"], t["z"][:, a:b].contiguous()]
    whole, h_end, _ = gdn.gdn_scan_fwd(*cut(0, 40), t["h0"])
    y, h, _ = gdn.gdn_scan_fwd(*cut(0, 37), t["h0"])
    ys = [y]
    for i in range(37, 40):
        y, h2, _ = gdn.gdn_scan_fwd(*cut(i, i + 1), h, h_T=h)
        assert h2 is h
        ys.append(y)
    assert R.rel(torch.cat(ys, 1), whole) <= 1e-6 and R.rel(h, h_end) <= 1e-6


# ---------------------------------------------------------------------------------- norm
NORM = [
    # M, G, D, dtype, pad, gate, act, center, w and b
    (1, 1, 1, "f32", 0, False, "none", True, True),
    (1, 4, 64, "bf16", 0, True, "silu", True, True),
    (3, 5, 24, "f32", 0, True, "silu", True, True),
    (70, 3, 37, "bf16", 0, False, "silu", True, True),
    (65, 2, 128, "bf16", 8, True, "silu", True, True),
    (33, 7, 192, "bf16", 0, True, "gelu", False, True),
    (129, 1, 256, "f32", 4, True, "silu", True, True),
    (20, 2, 256, "bf16", 3, False, "gelu", True, True),
    (40, 3, 512, "bf16", 0, True, "none", False, True),
    (11, 2, 512, "f32", 2, True, "silu", True, False),
    (9, 2, 513, "f32", 0, True, "silu", True, True),
    (70, 1, 2000, "bf16", 0, False, "silu", False, True),
    (1000, 2, 64, "f32", 0, False, "none", True, True),
]


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm(gdn, case):
    M, G, D, dtype, pad, gate, act, center, full = case
    r = Draw(M + G + D, dtype)
    C = G * D
    t = dict(x=r.wide(1, M, C, pad, pad)[0], w=1 + r.normal(C, scale=0.3, dtype=torch.float32) if full else None,
             b=r.normal(C, dtype=torch.float32) if full else None, z=r.wide(1, M, C, pad, 0)[0] if gate else None)
    dy = r.normal(M, C)
    y, stats = gdn.gdn_norm_fwd(t["x"], G, t["w"], t["b"], t["z"], act=act, center=center)
    d = gdn.gdn_norm_bwd(t["x"], G, stats, dy, t["w"], t["b"], t["z"], act=act, center=center)
    (y64,), g = R.with_grads(lambda x, w, b, z: R.norm(x, G, w, b, z, act, 1e-5, center), {k: d64(v) for k, v in t.items()},
                             (d64(dy),))
    if D == 1:                                          # x - mean is 0: y = act(b), and no gradient reaches x
        assert not d["dx"].any()
        g.pop("x")
    check("norm", {"y": y, **d}, {"y": y64, **{"d" + k: v for k, v in g.items()}})
    y2, none = gdn.gdn_norm_fwd(t["x"], G, t["w"], t["b"], t["z"], act=act, center=center, want_stats=False)
    assert none is None and torch.equal(y, y2)


def test_norm_of_constant_rows(gdn):
    """A group without variance: xh is 0 and the output act(b), nothing overflows."""
    x = torch.full((5, 256), 3.0, device="cuda", dtype=torch.bfloat16)
    b = torch.linspace(-2, 2, 256, device="cuda")
    y, _ = gdn.gdn_norm_fwd(x, 2, None, b, act="silu")
    assert R.rel(y, R.act("silu", b.double()).expand(5, 256)) <= TOL[torch.bfloat16]


# ---------------------------------------------------------------------------------- linear
LINEAR = [
    # M, N, K, dtype, pad, act, bias, res
    (1, 1, 1, "f32", 0, "none", True, True),
    (1, 256, 512, "bf16", 0, "silu", True, False),
    (2, 100, 72, "bf16", 0, "gelu", True, True),
    (7, 33, 65, "bf16", 3, "silu", True, True),
    (16, 1000, 200, "bf16", 8, "none", False, True),
    (16, 37, 129, "f32", 0, "gelu", True, True),
    (17, 128, 64, "bf16", 0, "silu", False, False),
    (100, 264, 328, "bf16", 0, "gelu", True, True),
    (129, 257, 63, "bf16", 1, "silu", True, True),
    (130, 130, 130, "f32", 2, "silu", True, True),
    (256, 512, 1024, "bf16", 0, "none", True, False),
    (300, 136, 2056, "bf16", 8, "silu", True, True),
    (513, 385, 200, "f32", 0, "none", False, False),
    (1000, 520, 72, "bf16", 0, "gelu", True, True),
]


@pytest.mark.parametrize("case", LINEAR, ids=str)
def test_linear(gdn, case):
    M, N, K, dtype, pad, act, bias, res = case
    r = Draw(M + N + K, dtype)
    t = dict(x=r.wide(1, M, K, pad, pad)[0], W=r.wide(1, N, K, pad, 0, scale=K ** -0.5)[0], bias=r.normal(N) if bias else None,
             res=r.wide(1, M, N, pad, pad)[0] if res else None)
    dy = r.normal(M, N)
    y, pre = gdn.gdn_linear_fwd(t["x"], t["W"], t["bias"], t["res"], act=act, want_pre=True)
    d = gdn.gdn_linear_bwd(t["x"], t["W"], dy, None if act == "none" else pre, act=act)
    (y64,), g = R.with_grads(lambda x, W, bias, res: R.linear(x, W, bias, res, act), {k: d64(v) for k, v in t.items()}, (d64(dy),))
    pre64 = R.linear(d64(t["x"]), d64(t["W"]), d64(t["bias"]), None, "none")
    g.pop("res", None)                                  # dy itself
    check("linear", {"y": y, "pre": pre, **d}, {"y": y64, "pre": pre64, **{"d" + k: v for k, v in g.items()}})
    y2, none = gdn.gdn_linear_fwd(t["x"], t["W"], t["bias"], t["res"], act=act)
    assert none is None and torch.equal(y, y2)
    one = gdn.gdn_linear_bwd(t["x"], t["W"], dy, None if act == "none" else pre, act=act, want_dx=False, want_dbias=False)
    assert one["dx"] is None and one["dbias"] is None and torch.equal(one["dW"], d["dW"])


# ------------------------------------------------------------------------------ all of them
def _everything(gdn, stream=None):
    t, lens, dy, ds_T, act = conv_inputs(CONV[4])
    out = list(gdn.gdn_conv_fwd(t["x"], t["w"], t["bias"], t["s0"], lens, stream=stream))
    out += gdn.gdn_conv_bwd(t["x"], t["w"], dy, t["bias"], t["s0"], lens, ds_T, stream=stream).values()
    for case in (SCAN[7], SCAN[13]):
        t, lens, dy, dh_T = scan_inputs(case)
        args = [t[k] for k in ("u", "dt", "A_log", "B", "C", "D", "dt_bias", "z")]
        fwd = gdn.gdn_scan_fwd(*args, t["h0"], lens, want_ckpt=True, stream=stream)
        out += fwd[:2]
        out += gdn.gdn_scan_bwd(*args[:5], fwd[2], dy, *args[5:], lens, dh_T, stream=stream).values()
    r = Draw(4, "bf16")
    x, z, dy, w, b = r.normal(500, 384), r.normal(500, 384), r.normal(500, 384), r.normal(384, dtype=torch.float32), None
    y, stats = gdn.gdn_norm_fwd(x, 3, w, b, z, stream=stream)
    out += [y, stats] + list(gdn.gdn_norm_bwd(x, 3, stats, dy, w, b, z, stream=stream).values())
    for M in (3, 300):
        x, W, dy = r.normal(M, 200), r.normal(264, 200), r.normal(M, 264)
        y, pre = gdn.gdn_linear_fwd(x, W, act="silu", want_pre=True, stream=stream)
        out += [y, pre] + list(gdn.gdn_linear_bwd(x, W, dy, pre, act="silu", stream=stream).values())
    return [o for o in out if o is not None]


def test_deterministic_and_on_another_stream(gdn):
    first = _everything(gdn)
    again = _everything(gdn)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = _everything(gdn)                      # the current stream is the side stream
    other = torch.cuda.Stream()
    with torch.cuda.stream(side):
        passed = _everything(gdn, stream=side)          # and passed explicitly
    side.synchronize()
    del other
    for k, (a, b, c, d) in enumerate(zip(first, again, on_side, passed)):
        eq = lambda x, y: torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))  # noqa: E731
        assert eq(a, b) and eq(a, c) and eq(a, d), k


def test_refusals_reach_the_caller(gdn):
    x = torch.zeros(2, 5, 8, device="cuda")
    w = torch.zeros(8, 5, device="cuda")
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_conv_fwd(x, w)                          # five taps
    assert e.value.code == -3
    with pytest.raises(gdn.GdnError):
        gdn.gdn_conv_fwd(x, w[:, :4].contiguous(), act="gelu")
    with pytest.raises(gdn.GdnError):
        gdn.gdn_norm_fwd(x, 2, eps=0.0)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_scan_fwd(x, x, torch.zeros(8, 65, device="cuda"), torch.zeros(2, 5, 1, 65, device="cuda"),
                         torch.zeros(2, 5, 1, 65, device="cuda"))
    with pytest.raises(ValueError, match="expected cuda"):
        gdn.gdn_linear_fwd(x, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="workspace"):
        gdn.gdn_conv_bwd(x, w[:, :4].contiguous(), x, workspace=torch.zeros(1 << 20, dtype=torch.uint8))


# --------------------------------------------------------------- offsets beyond 32 bits, more forms
def test_rows_far_apart(gdn):
    """Slices of a tensor of more than 2^31 elements: row offsets beyond 32 bits."""
    wide = torch.empty(40000, 65536, device="cuda", dtype=torch.bfloat16)
    r = Draw(12, "bf16")
    far = slice(39990, 40000)
    x = wide[:, 65536 - 128:]
    x.copy_(r.normal(40000, 128))
    y, _ = gdn.gdn_norm_fwd(x, 2)
    check("norm", {"y": y[far]}, {"y": R.norm(d64(x[far]), 2, None, None, None, "silu", 1e-5, True)})
    taps = r.normal(128, 4, dtype=torch.float32)
    y, _ = gdn.gdn_conv_fwd(x[None], taps)
    ref, _ = R.conv(d64(x[None, 39980:]), d64(taps), None, None, None, "silu")
    check("conv", {"y": y[:, far]}, {"y": ref[:, -10:]})
    W = r.normal(72, 128)
    y, _ = gdn.gdn_linear_fwd(x, W)
    check("linear", {"y": y[far]}, {"y": R.linear(d64(x[far]), d64(W), None, None, "none")})
    u, B, C = x[None, :, :64], x[None, :, 64:80].unflatten(2, (1, 16)), x[None, :, 80:96].unflatten(2, (1, 16))
    A_log = torch.zeros(64, 16, device="cuda") + 1.0
    y, _, _ = gdn.gdn_scan_fwd(u, u, A_log, B, C)        # decays of about exp(-2): the last steps forget the rest
    part = [d64(t[:, 39900:]) for t in (u, B, C)]
    ref, _ = R.scan(part[0], part[0], d64(A_log), part[1], part[2], None, None, None, None, None)
    check("scan", {"y": y[:, far]}, {"y": ref[:, -10:]})


@pytest.mark.parametrize("case", [(30, 2, 1024, "bf16", 0, True, "silu", True, True), (17, 1, 4096, "bf16", 0, False, "gelu", True, True),
                                  (9, 1, 4096, "f32", 0, True, "silu", False, True), (21, 2, 700, "f32", 2, True, "silu", True, True),
                                  (40, 3, 66, "bf16", 2, True, "silu", True, True), (5, 1, 5000, "bf16", 0, True, "silu", True, True)], ids=str)
def test_norm_layouts(gdn, case):
    """Groups held by a whole CTA, pairs of channels, and groups beyond a CTA's registers."""
    test_norm(gdn, case)


@pytest.mark.parametrize("case", [(20, 3000, 40, "bf16", 0, "silu", True, True), (33, 70, 130, "f32", 0, "gelu", True, True),
                                  (64, 200, 136, "bf16", 0, "gelu", True, True), (600, 300, 2000, "bf16", 0, "silu", True, False),
                                  (257, 513, 129, "f32", 0, "none", True, True), (2600, 2056, 320, "bf16", 0, "none", False, False)], ids=str)
def test_linear_layouts(gdn, case):
    """Few rows in each of their paddings, tiles of several rounds with halves and edges, float32 runs."""
    test_linear(gdn, case)


def test_linear_gradient_against_differences(gdn):
    """dx and dW against central differences of the float64 definition along random directions."""
    r = Draw(21, "f32")
    x, W, dy = r.normal(65, 70), r.normal(50, 70, scale=0.12), r.normal(65, 50)
    _, pre = gdn.gdn_linear_fwd(x, W, act="gelu", want_pre=True)
    d = gdn.gdn_linear_bwd(x, W, dy, pre, act="gelu")
    f = lambda a, b: (R.linear(a, b, None, None, "gelu") * d64(dy)).sum().item()  # noqa: E731
    h = 1e-5
    for name, way in (("dx", d64(r.normal(65, 70))), ("dW", d64(r.normal(50, 70)))):
        step = (way * h, 0.0) if name == "dx" else (0.0, way * h)
        numeric = (f(d64(x) + step[0], d64(W) + step[1]) - f(d64(x) - step[0], d64(W) - step[1])) / (2 * h)
        scale = (torch.linalg.vector_norm(d64(d[name])) * torch.linalg.vector_norm(way)).item()
        assert abs((d64(d[name]) * way).sum().item() - numeric) <= 1e-5 * scale, name


def test_conv_and_norm_gradients_against_differences(gdn):
    r = Draw(22, "f32")
    h = 1e-5
    x, w, b, dy = r.normal(2, 30, 12), r.normal(12, 4), r.normal(12), r.normal(2, 30, 12)
    d = gdn.gdn_conv_bwd(x, w, dy, b, want_ds0=False)
    f = lambda **k: (R.conv(k["x"], k["w"], k["bias"], None, None, "silu")[0] * d64(dy)).sum().item()  # noqa: E731
    cases = [(f, d, dict(x=x, w=w, bias=b))]
    x, w, b, z, dn = r.normal(20, 96), r.normal(96), r.normal(96), r.normal(20, 96), r.normal(20, 96)
    _, stats = gdn.gdn_norm_fwd(x, 4, w, b, z)
    g = lambda **k: (R.norm(k["x"], 4, k["w"], k["b"], k["z"], "silu", 1e-5, True) * d64(dn)).sum().item()  # noqa: E731
    cases.append((g, gdn.gdn_norm_bwd(x, 4, stats, dn, w, b, z), dict(x=x, w=w, b=b, z=z)))
    for fn, grads, leaves in cases:
        leaves = {k: d64(v) for k, v in leaves.items()}
        for k, v in leaves.items():
            way = d64(r.normal(*v.shape))
            numeric = (fn(**{**leaves, k: v + h * way}) - fn(**{**leaves, k: v - h * way})) / (2 * h)
            got = d64(grads["d" + k])
            scale = (torch.linalg.vector_norm(got) * torch.linalg.vector_norm(way)).item()
            assert abs((got * way).sum().item() - numeric) <= 1e-5 * scale, k


def test_in_a_cuda_graph(gdn):
    """The calls capture into a graph (caller's buffers, nothing allocated by the library) and replay."""
    r = Draw(30, "bf16")
    x, w = r.normal(4, 1, 256), r.normal(256, 4, dtype=torch.float32)
    W, s0, h0 = r.normal(264, 256, scale=0.06), r.normal(4, 3, 256), r.normal(4, 256, 16, dtype=torch.float32)
    A_log, bc = r.normal(256, 16, dtype=torch.float32), r.normal(4, 1, 1, 16)

    def step(s, h):
        a, _ = gdn.gdn_linear_fwd(x, W, act="silu")
        b, _ = gdn.gdn_conv_fwd(a[..., :256], w, None, s, s_T=s)
        c, _, _ = gdn.gdn_scan_fwd(b, b, A_log, bc, bc, h0=h, h_T=h)
        return gdn.gdn_norm_fwd(c, 4, want_stats=False)[0]

    s1, h1 = s0.clone(), h0.clone()
    want = [step(s1, h1) for _ in range(3)]
    s2, h2 = s0.clone(), h0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s2, h2)                                    # warm up: first calls set kernel attributes
    torch.cuda.current_stream().wait_stream(side)
    s2.copy_(s0)
    h2.copy_(h0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(s2, h2)
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k]), k
    assert torch.equal(s2, s1) and torch.equal(h2, h1)

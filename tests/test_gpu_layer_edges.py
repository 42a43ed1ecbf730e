"""The layer operators at the edges of what they take: the largest and the most awkward sizes,
states and values that are not finite, single rows at any address. References and tolerances are
those of test_gpu_layer.py."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layer_reference as R  # noqa: E402
from test_gpu_layer import TOL, Draw, check, clean, d64, gdn, scan_inputs  # noqa: E402,F401

F32, BF16 = torch.float32, torch.bfloat16


def same(a, b):
    """Equal values, NaN (of any payload) equal to NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(nan=0.0, posinf=float("inf"), neginf=float("-inf")),
                                                                       b.nan_to_num(nan=0.0, posinf=float("inf"), neginf=float("-inf")))


def test_the_most_rows(gdn):  # noqa: F811
    """The largest number of rows: 32-bit counters that end near 2^31."""
    n = 2 ** 31 - 65537
    r = Draw(1, "bf16")
    x = torch.empty(n, 1, dtype=BF16, device="cuda")
    x.view(-1).copy_(r.normal(1 << 20).repeat(2048)[:n])
    dy = x.flip(0)
    at = [slice(0, 2000), slice(n // 2, n // 2 + 2000), slice(n - 2000, n)]
    y, stats = gdn.gdn_norm_fwd(x, 1, act="silu", center=False)
    d = gdn.gdn_norm_bwd(x, 1, stats, dy, act="silu", center=False)
    for s in at:
        (y64,), g = R.with_grads(lambda x: R.norm(x, 1, None, None, None, "silu", 1e-5, False), {"x": d64(x[s])}, (d64(dy[s]),))
        check("norm", {"y": y[s]}, {"y": y64})
        # dx cancels to x * eps / (x^2 + eps)^1.5: its error is that of its two terms
        assert ((d["dx"][s].double() - g["x"]).abs() <= 2 ** -8 * g["x"].abs() + 1e-5 * d64(dy[s] / x[s]).abs()).all()
    del y, stats, d
    taps = r.normal(1, 4, dtype=F32)
    y, s_T = gdn.gdn_conv_fwd(x[None], taps)
    d = gdn.gdn_conv_bwd(x[None], taps, dy[None], want_ds0=False)
    for s in at[1:]:
        wide = slice(s.start - 6, s.stop)
        (y64, s64), g = R.with_grads(lambda x: R.conv(x, d64(taps), None, None, None, "silu"), {"x": d64(x[None, wide])}, (d64(dy[None, wide]), None))
        check("conv", {"y": y[:, s]}, {"y": y64[:, 6:]})
        inner = slice(3, 2000 + 6 - (0 if s.stop == n else 3))
        check("conv", {"dx": d["dx"][:, wide][:, inner]}, {"dx": g["x"][:, inner]})
    assert torch.equal(s_T[0], x[-3:])


@pytest.mark.parametrize("C", [2097152 + 1, 4194303])
def test_conv_of_more_channel_blocks_than_an_axis_of_the_grid(gdn, C):  # noqa: F811
    r = Draw(2, "bf16")
    x, w, dy = r.normal(1, 2, C), r.normal(C, 2, dtype=F32), r.normal(1, 2, C)
    y, s_T = gdn.gdn_conv_fwd(x, w, act="none")
    d = gdn.gdn_conv_bwd(x, w, dy, act="none", want_ds0=False)
    (y64, s64), g = R.with_grads(lambda x, w: R.conv(x, w, None, None, None, "none"), {"x": d64(x), "w": d64(w)}, (d64(dy), None))
    check("conv", {"y": y, "s_T": s_T, **d}, {"y": y64, "s_T": s64, "dx": g["x"], "dw": g["w"]})


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_conv_state_that_is_not_finite(gdn, bad, act):  # noqa: F811
    """The state of a row without valid steps takes no part in the parameters' gradients, and that of a
    row of one step only through that step."""
    r = Draw(3, "bf16")
    lens = torch.tensor([9, 0, 1], dtype=torch.int32, device="cuda")
    t = dict(x=r.normal(3, 9, 24), w=r.normal(24, 4, dtype=F32), bias=r.normal(24, dtype=F32), s0=r.normal(3, 3, 24))
    dy, ds_T = r.normal(3, 9, 24), r.normal(3, 3, 24)
    t["s0"][1] = bad
    t["s0"][2, 2, :8] = bad
    d = gdn.gdn_conv_bwd(t["x"], t["w"], dy, t["bias"], t["s0"], lens, ds_T, act=act)
    leaves = {k: d64(clean(v, lens) if k == "x" else v) for k, v in t.items()}
    leaves["s0"][1] = 0.0
    _, g = R.with_grads(lambda x, w, bias, s0: R.conv(x, w, bias, s0, lens, act), leaves, (d64(clean(dy, lens)), d64(ds_T)))
    assert torch.isfinite(d["dw"][8:]).all() and torch.isfinite(d["dbias"][8:]).all()
    check("conv", d, {"d" + k: v for k, v in g.items()})


@pytest.mark.parametrize("T", [1, 16, 40, 1030])
@pytest.mark.parametrize("which", ["h0", "dh_T"])
def test_scan_state_of_a_row_without_steps(gdn, T, which):  # noqa: F811
    """A state (or its cotangent) that is not finite in a row without valid steps passes through and
    takes no part in any gradient. (T = 1030 is split into segments.)"""
    t, lens, dy, dh_T = scan_inputs((3, T, 24, 8, 2, "f32", 0, True, [T, 0, (T + 1) // 2], True, True))
    bad = t["h0"] if which == "h0" else dh_T
    bad[1], bad[1, ::2] = float("nan"), float("inf")
    order = ("u", "dt", "A_log", "B", "C", "D", "dt_bias", "z")
    args = [t[k] for k in order]
    y, h_T, ckpt = gdn.gdn_scan_fwd(*args, t["h0"], lens, want_ckpt=True)
    d = gdn.gdn_scan_bwd(*args[:5], ckpt, dy, *args[5:], lens, dh_T)
    assert same(h_T[1], t["h0"][1]) and not y[1].any() and same(d["dh0"][1], dh_T[1])
    keep = bad.clone()
    keep[1] = 0.0
    leaves = {k: d64(clean(v, lens) if k in ("u", "dt", "B", "C", "z") else v) for k, v in t.items()}
    cot = [dy, dh_T]
    if which == "h0":
        leaves["h0"] = d64(keep)
    else:
        cot[1] = keep
    _, g = R.with_grads(lambda **k: R.scan(lens=lens, **k), leaves, (d64(clean(cot[0], lens)), d64(cot[1])))
    g["h0"][1] = d64(dh_T[1])
    check("scan grads", d, {"d" + k: v for k, v in g.items()})


def test_scan_gradients_behind_a_row_are_zeros(gdn):  # noqa: F811
    """Zeros behind the valid steps, also where the row's own state is not finite."""
    t, lens, dy, dh_T = scan_inputs((2, 75, 40, 32, 1, "f32", 0, True, [75, 35], True, True))
    t["h0"][1] = float("nan")
    args = [t[k] for k in ("u", "dt", "A_log", "B", "C", "D", "dt_bias", "z")]
    y, _, ckpt = gdn.gdn_scan_fwd(*args, t["h0"], lens, want_ckpt=True)
    d = gdn.gdn_scan_bwd(*args[:5], ckpt, dy, *args[5:], lens, dh_T)
    for out in (y, *(d[k] for k in ("du", "ddt", "dB", "dC", "dz"))):
        assert not out[1, 35:].any() and torch.isfinite(out[0]).all()
    assert torch.isnan(y[1, :35]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(1, 24), (1, 1), (5, 1), (64, 1), (1, 700)])
def test_linear_single_rows_at_any_address(gdn, M, N, dtype):  # noqa: F811
    """A slice with one row counts as contiguous, wherever it begins. (With an activation the bf16 rounding of
    a single pre-activation would be scaled by the slope's condition: float32 only.)"""
    r, act = Draw(5, dtype), "silu" if dtype == "f32" else "none"
    for K in (40, 41):
        x, W, dy, bias, res = r.normal(M, 200)[:, 3:3 + K], r.normal(N, 200)[:, 5:5 + K], r.normal(M, N), r.normal(N), r.normal(M, 1000)[:, 1:1 + N]
        y, pre = gdn.gdn_linear_fwd(x, W, bias, res, act=act, want_pre=True)
        d = gdn.gdn_linear_bwd(x, W, dy, pre, act=act)
        leaves = dict(x=d64(x), W=d64(W), bias=d64(bias))
        (y64,), g = R.with_grads(lambda x, W, bias: R.linear(x, W, bias, d64(res), act), leaves, (d64(dy),))
        check("linear", {"y": y, **d}, {"y": y64, **{"d" + k: v for k, v in g.items()}})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(3, 24, 40), (16, 8, 24), (32, 70, 33)])
def test_linear_few_packed_rows_at_any_address(gdn, M, N, K, dtype):  # noqa: F811
    r = Draw(6, dtype)
    x, W = r.normal(M * K + 1)[1:].view(M, K), r.normal(N * K + 1)[1:].view(N, K)
    y, _ = gdn.gdn_linear_fwd(x, W)
    check("linear", {"y": y}, {"y": d64(x) @ d64(W).t()})
    if dtype == "f32":
        dy = r.normal(M, N)
        check("linear", gdn.gdn_linear_bwd(x, W, dy), {"dx": d64(dy) @ d64(W), "dW": d64(dy).t() @ d64(x)})
    else:
        with pytest.raises(gdn.GdnError) as e:          # the gradients' products read bf16 rows in place
            gdn.gdn_linear_bwd(x, W, r.normal(M, N))
        assert e.value.code == -2


@pytest.mark.parametrize("tail", [0x007f7f, 0x008080, 0x00ff7f, 0x7fffff, None])
def test_linear_float32_products_hold_24_bits(gdn, tail):  # noqa: F811
    """One product per output, so that nothing averages out: the terms that the tensor cores' form of
    float32 drops are below 2^-23.9 of it, its last addition cuts less than 2^-23: 2^-22 in all."""
    r = Draw(7, "f32")

    def values(n):
        v = torch.rand(n, device="cuda", generator=r.g) + 1
        v = v if tail is None else (v.view(torch.int32) & ~0xffff | tail).view(F32)
        return v * torch.sign(torch.randn(n, device="cuda", generator=r.g))

    M, N, K = 300, 200, 70
    x, W, dy = torch.zeros(M, K, device="cuda"), torch.zeros(N, K, device="cuda"), torch.zeros(M, N, device="cuda")
    x[:, 3], W[:, 3], dy[:, 5] = values(M), values(N), values(M)
    y, _ = gdn.gdn_linear_fwd(x, W)
    assert ((d64(y) - d64(x) @ d64(W).t()).abs() <= 2.0 ** -22 * (d64(x) @ d64(W).t()).abs()).all()
    W[5] = values(K)
    dx = gdn.gdn_linear_bwd(x, W, dy)["dx"]
    ref = d64(dy) @ d64(W)
    assert ((d64(dx) - ref).abs() <= 2.0 ** -22 * ref.abs()).all()


def test_linear_float32_of_the_largest_values(gdn):  # noqa: F811
    """Values that bf16 would round to infinity."""
    top = torch.finfo(F32).max
    x, W = torch.zeros(64, 40, device="cuda"), torch.zeros(48, 40, device="cuda")
    x[:, 0] = torch.linspace(0.9, 1.0, 64, device="cuda") * top
    x[1::2] *= -1
    W[:, 0] = torch.linspace(0.1, 0.99, 48, device="cuda")
    y, _ = gdn.gdn_linear_fwd(x, W)
    assert R.rel(y, d64(x) @ d64(W).t()) <= TOL[F32]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(4, 50, 70), (64, 50, 70), (300, 130, 72), (300, 130, 700)])
def test_linear_infinities(gdn, M, N, K, dtype):  # noqa: F811
    """Infinities and NaN where the definition has them, whatever the number of rows: an infinity by a
    value of few bits, by its opposite, by zero, by another infinity."""
    r = Draw(8, dtype)
    x, W, dy = r.normal(M, K), r.normal(N, K, scale=K ** -0.5), r.normal(M, N)
    W[:, :40] = torch.sign(W[:, :40])                   # nothing in the second and third terms
    inf = float("inf")
    x[0, 5], x[1, 6], x[2, 50], x[3, 1], x[3, 2] = inf, -inf, inf, inf, inf
    W[4, 5], W[7, 11], W[9, 5] = 0.0, inf, -inf
    dy[1, 3], dy[2, 8] = inf, float("nan")
    y, _ = gdn.gdn_linear_fwd(x, W)
    d = gdn.gdn_linear_bwd(x, W, dy)
    for got, ref in ((y, d64(x) @ d64(W).t()), (d["dx"], d64(dy) @ d64(W)), (d["dW"], d64(dy).t() @ d64(x))):
        for f in (torch.isnan, torch.isposinf, torch.isneginf):
            assert torch.equal(f(got), f(ref)), f
        assert R.rel(got, ref) <= TOL[got.dtype]


def test_parameter_gradients_that_overflow(gdn):  # noqa: F811
    """Sums over rows that hold an infinity are that infinity, in every operator's parameter gradients."""
    r = Draw(9, "f32")
    inf = float("inf")

    def expect(got, ref):
        for f in (torch.isnan, torch.isposinf, torch.isneginf):
            assert torch.equal(f(got), f(ref)), f
        assert R.rel(got, ref) <= TOL[F32]

    dy = r.normal(300, 48)
    dy[7, 3], dy[9, 4], dy[11, 5], dy[12, 5], dy[13, 6] = inf, -inf, inf, -inf, float("nan")
    x, W = r.normal(300, 40), r.normal(48, 40)
    expect(gdn.gdn_linear_bwd(x, W, dy, want_dx=False)["dbias"], d64(dy).sum(0))
    xn, b = r.normal(300, 48), r.normal(48)
    _, stats = gdn.gdn_norm_fwd(xn, 3, None, b, act="none")
    expect(gdn.gdn_norm_bwd(xn, 3, stats, dy, None, b, act="none")["db"], d64(dy).sum(0))
    xc, w = r.normal(1, 300, 48), r.normal(48, 4)
    expect(gdn.gdn_conv_bwd(xc, w, dy[None], act="none", want_ds0=False)["dbias"], d64(dy).sum(0))
    u, A_log, bc, D = torch.ones(1, 300, 48, device="cuda"), r.normal(48, 8), r.normal(1, 300, 1, 8), r.normal(48)
    _, _, ckpt = gdn.gdn_scan_fwd(u, u, A_log, bc, bc, D, want_ckpt=True)
    expect(gdn.gdn_scan_bwd(u, u, A_log, bc, bc, ckpt, dy[None], D)["dD"], d64(dy).sum(0))


def _one_sign(r, *shape):
    return (torch.rand(*shape, device="cuda", generator=r.g) + 1).to(BF16)


def _product64(a, b):
    """a b^T of [M, K] and [N, K], by parts of K."""
    return sum(d64(x) @ d64(y).t() for x, y in zip(a.split(1 << 18, 1), b.split(1 << 18, 1)))


def test_linear_gradient_of_many_rows(gdn):  # noqa: F811
    """4e6 rows of one sign: the tensor cores' accumulation, which truncates, alone would lose 2.4 %."""
    r = Draw(10, "bf16")
    x, dy, W = _one_sign(r, 4000000, 64), _one_sign(r, 4000000, 64), r.normal(64, 64)
    d = gdn.gdn_linear_bwd(x, W, dy, want_dx=False)
    check("many rows", d, {"dW": _product64(dy.t(), x.t()), "dbias": dy.double().sum(0)})


@pytest.mark.parametrize("M,N,K,act", [(70, 40, 2000000, "none"), (300, 520, 70008, "silu"), (64, 72, 70000, "gelu"), (64, 72, 540000, "none"),
                                       (16, 256, 100000, "none"), (7, 100, 540000, "silu"), (2600, 2056, 65600, "none"),
                                       (260, 130, 65537, "silu")], ids=str)
def test_linear_long_sums(gdn, M, N, K, act):  # noqa: F811
    """Products over long K in several runs: partial sums in whole, half and edge tiles, in both gradients
    (over M and over N), and in the decode forms."""
    r = Draw(11, "bf16")
    x, W, bias, res = _one_sign(r, M, K), _one_sign(r, N, K) / K, r.normal(N), r.normal(M, N)
    y, pre = gdn.gdn_linear_fwd(x, W, bias, res, act=act, want_pre=True)
    core = _product64(x, W)
    check("long", {"y": y, "pre": pre}, {"y": R.act(act, core + d64(bias)) + d64(res), "pre": core + d64(bias)})
    # the same sizes as gradients: K rows give dW, K outputs give dx
    dy, a = _one_sign(r, K, N), _one_sign(r, K, M)
    dW = gdn.gdn_linear_bwd(a, r.normal(N, M), dy, want_dx=False, want_dbias=False)["dW"]
    check("long dW", {"dW": dW}, {"dW": _product64(dy.t(), a.t())})
    if M * K < 1 << 27:
        dy, Wl = _one_sign(r, M, K), _one_sign(r, K, N)
        dx = gdn.gdn_linear_bwd(r.normal(M, N), Wl, dy, want_dW=False, want_dbias=False)["dx"]
        check("long dx", {"dx": dx}, {"dx": _product64(dy, Wl.t())})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [3, 63, 100, 168, 700, 1025, 5000])
def test_norm_of_large_constant_groups(gdn, D, dtype):  # noqa: F811
    """Groups of equal values far from 0 (their sums are exact in float32): no variance, xh is 0 and the
    output act(b). A mean that is an ulp off would give xh up to 0.02."""
    c = torch.arange(128, 256, device="cuda").float() * 4                 # 512 to 1020
    x = c[:, None].expand(128, 2 * D).contiguous().to(Draw(1, dtype).dtype)
    b = torch.linspace(-2, 2, 2 * D, device="cuda")
    y, stats = gdn.gdn_norm_fwd(x, 2, None, b, act="silu")
    check("norm", {"y": y}, {"y": R.act("silu", b.double()).expand(128, 2 * D)})
    assert torch.equal(stats[..., 0], c[:, None].expand(128, 2))


@pytest.mark.parametrize("case", [(3, 1, 24, 32, 1, "bf16", 0, True, None, True, True), (5, 1, 18, 23, 2, "f32", 0, True, [1, 0, 1, 1, 0], True, True),
                                  (2, 1, 40, 64, 1, "f32", 0, True, None, False, True), (6, 1, 20, 49, 2, "bf16", 8, True, None, True, False),
                                  (9, 1, 35, 20, 5, "bf16", 3, False, [1, 1, 0, 1, 1, 0, 1, 1, 1], True, True)], ids=str)
def test_scan_steps_of_many_states(gdn, case):  # noqa: F811
    """Single steps where 8 or 16 lanes share a channel, and their state updated in place."""
    t, lens, _, _ = scan_inputs(case)
    args = [t[k] for k in ("u", "dt", "A_log", "B", "C", "D", "dt_bias", "z")]
    y, h, _ = gdn.gdn_scan_fwd(*args, t["h0"], lens)
    y64, h64 = R.scan(lens=lens, **{k: d64(clean(v, lens) if k in ("u", "dt", "B", "C", "z") else v) for k, v in t.items()})
    check("scan", {"y": y, "h_T": h}, {"y": y64, "h_T": h64})
    if t["h0"] is not None:
        y2, h2, _ = gdn.gdn_scan_fwd(*args, t["h0"], lens, h_T=t["h0"])
        assert h2 is t["h0"] and torch.equal(h2, h) and torch.equal(y2, y)

"""The norms around a block on the GPU against their float64 definition: forward and gradients, every form
(with and without either norm, gates for each row or shared, activations), row lengths and layouts.

Tolerances (2-norm): bf16 outputs are off by at most 2^-8 of themselves, float32 ones by some roundings of
2^-24 (about ten in a row's chain and the sums over channels and rows, of either sign: 2^-24 x 16).

The gradient through a norm, rstd (f - hh mean(f hh)), is a difference: each term carries up to eight
roundings of 2^-24 of f, so dh is off by up to 2^-21 of |rstd f| besides, and dx by as much of |rstd e|,
e = dy w_pre, with what follows from it. That counts where the terms cancel: with one channel hh^2 = 1 - eps rstd^2, dh = rstd f eps rstd^2, and the difference keeps 2^-21 / (eps
rstd^2), some 5e-2, of it at eps = 1e-5 and h of order 1 (measured: 1.2e-2), whatever the order of the sums in
float32."""
import pytest

torch = pytest.importorskip("torch")
import block_reference as K  # noqa: E402
import layer_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TOL = {F32: 16 * 2 ** -24, BF16: 2 ** -8}
LEAVES = ("x", "h", "z", "scale", "w_post", "w_pre")


def gdn():
    import gated_delta_rule_22_gb300
    return gated_delta_rule_22_gb300


def make(seed, lead, D, dt, gate, scale=True, weights=True, post=True, pre=True, wide=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    rows = lambda *s: rnd(*s, D).to(dt) if not wide else rnd(*s, D + wide).to(dt)[..., wide // 2:wide // 2 + D]  # noqa: E731
    a = dict(x=rows(*lead), h=rows(*lead), z=None if gate is None else rows(*lead[:gate]), scale=rnd(D) * 0.3 if scale else None,
             w_post=1 + 0.2 * rnd(D) if weights and post else None, w_pre=1 + 0.2 * rnd(D) if weights and pre else None,
             dy=rnd(*lead, D).to(dt) if pre else None, dr=rnd(*lead, D).to(dt))
    return a


def check(a, post=True, pre=True, act="none", dr=True, eps=1e-5):
    f = lambda **kw: K.resnorm(**kw, post=post, pre=pre, act=act, eps=eps)  # noqa: E731
    cot = [a["dr"].double() if dr else torch.zeros_like(a["x"], dtype=torch.float64)] + ([a["dy"].double()] if pre else [])
    outs, grads = R.with_grads(f, {n: None if a[n] is None else a[n].double() for n in LEAVES}, cot)
    form = dict(post=post, pre=pre, act=act, eps=eps)
    params = (a["z"], a["scale"], a["w_post"], a["w_pre"])
    r, y, stats = gdn().gdn_resnorm_fwd(a["x"], a["h"], *params, **form)
    d = gdn().gdn_resnorm_bwd(a["x"], a["h"], stats, a["dy"], a["dr"] if dr else None, *params, **form)
    torch.cuda.synchronize()
    got = {"r": (r, outs[0])}
    if pre:
        got["y"] = (y, outs[1])
    else:
        assert y is None
    for n in LEAVES:
        if a[n] is None:
            assert d["d" + n] is None
        else:
            got["d" + n] = (d["d" + n], grads[n])
    f = grads["x"]
    for n in ("scale", "w_post"):
        f = f if a[n] is None else f * a[n].double()
    if a["z"] is not None:
        gate = R.act(act, a["z"].double())
        f = f * gate.reshape(gate.shape[:-1] + (1,) * (f.dim() - gate.dim()) + gate.shape[-1:])
    if post:
        f = f / torch.sqrt((a["h"].double() ** 2).mean(-1, keepdim=True) + eps)
    lost_r = 0.0                                       # of dx by the norm in front, relative
    if pre:
        e = a["dy"].double() / torch.sqrt((outs[0] ** 2).mean(-1, keepdim=True) + eps)
        e = e if a["w_pre"] is None else e * a["w_pre"].double()
        lost_r = 2 ** -21 * (e.norm() / grads["x"].norm()).item()
    for n, (mine, ref) in got.items():
        assert mine.shape == ref.shape
        tol = TOL[mine.dtype] + (lost_r if n in ("dx", "dh", "dz", "dscale", "dw_post") else 0.0)
        tol += 2 ** -21 * (f.norm() / ref.norm()).item() * (1 + lost_r) if n == "dh" else 0.0
        assert R.rel(mine, ref) <= tol, (n, R.rel(mine, ref))
    return r, y, stats, d


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 64, 72, 255, 256, 264, 1000, 1024, 1030, 2048, 2056, 4096, 5000, 8192, 8200, 12289, 16384])
def test_row_lengths(D, dt):
    check(make(1, (3, 5), D, dt, 2), act="silu")
    check(make(2, (7,), D, dt, None))


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", [None, 0, 1, 2])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_forms(post, pre, gate, dt):
    for i, act in enumerate(("none", "silu", "gelu")):
        for scale, weights in ((True, True), (False, False)):
            check(make(10 + i, (4, 37), 192, dt, gate, scale, weights, post, pre), post, pre, act)
    if pre:
        check(make(20, (4, 37), 192, dt, gate, True, True, post, pre), post, pre, "silu", dr=False)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lead,gate,D", [((1, 3000), 1, 64), ((2000, 2), 1, 40), ((70000, 2), 1, 8), ((1300, 1), 1, 264), ((3, 700), 1, 520),
                                         ((5000,), None, 96), ((1,), 0, 2048), ((2, 3, 50), 2, 128), ((2, 3, 50), 1, 128)])
def test_rows_and_shared_gates(lead, gate, D, dt):
    check(make(3, lead, D, dt, gate), act="silu")


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("wide", [16, 2, 1])
def test_column_slices(wide, dt):
    check(make(4, (3, 41), 200, dt, 2, wide=wide), act="silu")
    check(make(5, (3, 41), 1000, dt, 1, wide=wide), act="silu")


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 1000, 2048, 9000])
def test_stream_updated_in_place(D, dt):
    a = make(6, (300,), D, dt, None)
    r, y, _ = gdn().gdn_resnorm_fwd(a["x"], a["h"], None, a["scale"], a["w_post"], a["w_pre"])
    x = a["x"].clone()
    r2, y2, stats = gdn().gdn_resnorm_fwd(x, a["h"], None, a["scale"], a["w_post"], a["w_pre"], r=x, want_stats=False)
    assert r2 is x and stats is None and torch.equal(r, x) and torch.equal(y, y2)


def test_rows_of_zeros_and_large_values():
    a = make(7, (6,), 256, F32, None)
    a["h"][2] = 0.0
    a["x"][3] = 0.0
    a["h"][3] = 0.0
    a["x"][4] *= 1e15
    check(a)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_a_row_that_is_not_finite_stays_by_itself(dt):
    a = make(8, (40,), 512, dt, None)
    whole = gdn().gdn_resnorm_fwd(a["x"], a["h"], None, a["scale"], a["w_post"], a["w_pre"])
    a["h"][7, 3] = float("nan")
    r, y, _ = gdn().gdn_resnorm_fwd(a["x"], a["h"], None, a["scale"], a["w_post"], a["w_pre"])
    keep = torch.arange(40, device="cuda") != 7
    assert torch.equal(r[keep], whole[0][keep]) and torch.equal(y[keep], whole[1][keep]) and y[7].isnan().all()


@pytest.mark.parametrize("gate", [None, 1, 2])
def test_deterministic_captured_and_on_a_stream(gate):
    a, b = make(9, (4, 600), 1024, BF16, gate), make(10, (4, 600), 1024, BF16, gate)

    def run(s, stream=None):
        p = (s["z"], s["scale"], s["w_post"], s["w_pre"])
        r, y, stats = gdn().gdn_resnorm_fwd(s["x"], s["h"], *p, act="silu", stream=stream)
        d = gdn().gdn_resnorm_bwd(s["x"], s["h"], stats, s["dy"], s["dr"], *p, act="silu", stream=stream)
        return [t for t in (r, y, stats, *d.values()) if t is not None]

    first, other = run(a), run(b)
    assert all(torch.equal(x, y) for x, y in zip(first, run(a)))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    onstream = run(a, s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, onstream))
    live = {n: None if t is None else t.clone() for n, t in a.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(live)
    for want, src in ((first, a), (other, b)):
        for n, t in live.items():
            if t is not None:
                t.copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out))


def test_gradients_against_differences():
    """Central differences of the float32 forward along a direction: the loss is of order 100, its rounding
    2^-24 x 100 x a few over a step of 2 x 0.01, and the third derivative's share some 1e-4: 2e-3 of the
    gradient's size."""
    a = make(11, (3, 20), 96, F32, 1)
    p = lambda s: (s["z"], s["scale"], s["w_post"], s["w_pre"])  # noqa: E731
    _, _, stats = gdn().gdn_resnorm_fwd(a["x"], a["h"], *p(a), act="silu")
    d = gdn().gdn_resnorm_bwd(a["x"], a["h"], stats, a["dy"], a["dr"], *p(a), act="silu")
    for name in LEAVES:
        way = torch.randn_like(a[name])
        loss = []
        for sign in (1, -1):
            m = dict(a)
            m[name] = a[name] + sign * 0.01 * way
            r, y, _ = gdn().gdn_resnorm_fwd(m["x"], m["h"], *p(m), act="silu")
            loss.append((y.double() * a["dy"].double()).sum() + (r.double() * a["dr"].double()).sum())
        numeric, exact = ((loss[0] - loss[1]) / 0.02).item(), (way.double() * d["d" + name].double()).sum().item()
        assert abs(numeric - exact) <= 2e-3 * (abs(exact) + d["d" + name].norm().item()), name

"""Linear attention with a decay and the norms around a block on the GPU: calls of the C ABI that the binding
does not make, and what the header says of one row, one prompt or one input beside the others."""
import ctypes
import random

import pytest

torch = pytest.importorskip("torch")
import block_reference as K  # noqa: E402
import layer_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gdn():
    import gated_delta_rule_22_gb300
    return gated_delta_rule_22_gb300


def _at(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def resnorm_bwd_abi(a, stats, gate_rows, z=None, want_dz=True):
    """gdn_resnorm_bwd as a C program calls it, outputs preset to NaN with rows behind them; workspace of exactly
    the size asked for."""
    from gated_delta_rule_22_gb300 import layer as Ly
    M, D = a["x"].shape
    dt = a["x"].dtype
    shape = Ly.GdnResnormShape(M, D, gate_rows, 1, 1, 1, 1 if dt is BF16 else 0, 1e-5, 0, 0, 0)
    lib = Ly._library()
    need = lib.gdn_resnorm_bwd_workspace_bytes(ctypes.byref(shape))
    ws = torch.full((need + 256,), 0x7f, dtype=torch.uint8, device="cuda")
    rows = lambda n: torch.full((n + 3, D), float("nan"), dtype=dt, device="cuda")  # noqa: E731
    out = {"dx": rows(M), "dh": rows(M), "dz": rows(M // gate_rows) if z is not None and want_dz else None}
    out.update({n: torch.full((D,), float("nan"), device="cuda") for n in ("dscale", "dw_post", "dw_pre")})
    rc = lib.gdn_resnorm_bwd(ctypes.byref(shape), *map(_at, (a["x"], a["h"], z, a["scale"], a["w_post"], a["w_pre"], stats, a["dy"], a["dr"], out["dx"],
                                                             out["dh"], out["dz"], out["dscale"], out["dw_post"], out["dw_pre"], ws)), need,
                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    assert torch.all(ws[need:] == 0x7f)
    for n in ("dx", "dh", "dz"):
        if out[n] is not None:
            assert out[n][-3:].isnan().all(), n
            out[n] = out[n][:-3]
    return out


def resnorm_rows(seed, M, D, dt):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(x=rnd(M, D).to(dt), h=rnd(M, D).to(dt), scale=rnd(D) * 0.3, w_post=1 + 0.2 * rnd(D), w_pre=1 + 0.2 * rnd(D),
                dy=rnd(M, D).to(dt), dr=rnd(M, D).to(dt))


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,gate_rows,D", [(12, 3, 64), (8, 4, 33), (5, 5, 64), (4096, 1024, 96), (999, 333, 1030), (65536, 2, 8), (1, 1, 8)])
def test_resnorm_gradients_without_a_gate_at_any_gate_rows(M, gate_rows, D, dt):
    """gate_rows has no effect without z: the same bits as with 1, every row written, none behind the last. Against
    the definition: half a step of the outputs' type, and in float32 some roundings of 2^-24 (16 of either sign) and, through
    a norm's difference, 2^-21 of |rstd f| (with rstd of order 1 and |f| of |dh|'s order: 2^-20)."""
    a = resnorm_rows(M + D, M, D, dt)
    _, _, stats = gdn().gdn_resnorm_fwd(a["x"], a["h"], None, a["scale"], a["w_post"], a["w_pre"])
    got, one = resnorm_bwd_abi(a, stats, gate_rows), resnorm_bwd_abi(a, stats, 1)
    names = {"x": "dx", "h": "dh", "scale": "dscale", "w_post": "dw_post", "w_pre": "dw_pre"}
    assert all(torch.equal(got[n], one[n]) for n in names.values())
    f = lambda **kw: K.resnorm(z=None, **kw, post=True, pre=True, act="none", eps=1e-5)  # noqa: E731
    _, grads = R.with_grads(f, {n: a[n].double() for n in names}, (a["dr"].double(), a["dy"].double()))
    for n, d in names.items():
        tol = 2 ** -8 if got[d].dtype is BF16 else 16 * 2 ** -24 + 2 ** -20
        assert R.rel(got[d], grads[n]) <= tol, (d, R.rel(got[d], grads[n]))


@pytest.mark.parametrize("M,gate_rows", [(12, 3), (4096, 1024), (1000, 2)])
def test_resnorm_gradients_with_a_gate_whose_own_is_not_wanted(M, gate_rows):
    """dz NULL beside a z: the other outputs keep their bits."""
    a = resnorm_rows(M, M, 128, BF16)
    z = torch.randn(M // gate_rows, 128, device="cuda").to(BF16)
    x3, h3 = (a[n].view(M // gate_rows, gate_rows, 128) for n in "xh")
    _, _, stats = gdn().gdn_resnorm_fwd(x3, h3, z, a["scale"], a["w_post"], a["w_pre"], act="silu")
    with_dz, without = resnorm_bwd_abi(a, stats, gate_rows, z), resnorm_bwd_abi(a, stats, gate_rows, z, want_dz=False)
    assert without["dz"] is None and with_dz["dz"].isfinite().all()
    assert all(torch.equal(with_dz[n], without[n]) for n in with_dz if n != "dz")


def linattn_inputs(seed, B, T, Hk, Hv, Dk, Dv, dt, g=None):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s, scale=1.0: torch.randn(*s, generator=gen, device="cuda") * scale  # noqa: E731
    decay = torch.exp(-torch.exp2(-8.0 * (torch.arange(Hv, device="cuda") + 0.5) / Hv)) if g is None else torch.full((Hv,), g, device="cuda")
    return dict(q=rnd(B, T, Hk, Dk, scale=Dk ** -0.5).to(dt), k=rnd(B, T, Hk, Dk).to(dt), v=rnd(B, T, Hv, Dv).to(dt), g=decay, S0=rnd(B, Hv, Dv, Dk),
                dy=rnd(B, T, Hv, Dv).to(dt), dS_T=rnd(B, Hv, Dv, Dk, scale=0.3))


def linattn(a, train=True, rows=slice(None), state=True):
    a = {n: t if n == "g" else t[rows] for n, t in a.items()}
    S0, dS_T = (a["S0"], a["dS_T"]) if state else (None, None)
    out = dict(zip(("y", "S_T"), gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], S0)))
    if train:
        out.update(gdn().gdn_linattn_bwd(a["q"], a["k"], a["v"], a["g"], a["dy"], S0, None, dS_T))
    return out


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 5, 600])
def test_linattn_rows_beside_others_and_alone(T, dt):
    """40 rows of 4 heads fill the SMs and go whole, one goes in segments: a row's results differ by what both are
    off the definition at most (twice 1.5 x 2^-8 in bf16, twice 4e-6 in float32, states twice 2^-20). A single step has no
    segments: the same bits."""
    a = linattn_inputs(1, 40, T, 2, 4, 64, 64, dt)
    whole = linattn(a)
    for b in (0, 17, 39):
        for n, x in linattn(a, rows=slice(b, b + 1)).items():
            if T == 1 and n in ("y", "S_T"):
                assert torch.equal(x[0], whole[n][b]), n
            else:
                tol = 2 ** -19 if n in ("S_T", "dS0") else 3 * 2 ** -8 if dt is BF16 else 8e-6
                assert R.rel(x[0], whole[n][b].double()) <= tol, (n, b, R.rel(x[0], whole[n][b].double()))


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate", [None, "sequence", "step"])
def test_resnorm_rows_beside_others_and_alone(gate, dt):
    """The same bits for a batch and for its rows one by one, but for the gradient of a gate that a sequence's steps
    share, whose units are cut by the number of sequences: sums of 700 float32 terms of either sign in two orders (each off
    by a few 2^-24 of them), rounded once."""
    B, T, D = 6, 700, 192
    rows = resnorm_rows(3, B * T, D, dt)
    a = {n: t.view(B, T, D) if t.dim() == 2 else t for n, t in rows.items()}
    z = None if gate is None else torch.randn(*((B, D) if gate == "sequence" else (B, T, D)), device="cuda").to(dt)

    def run(s):
        x, h, dy, dr = (a[n][s] for n in ("x", "h", "dy", "dr"))
        p = (None if z is None else z[s], a["scale"], a["w_post"], a["w_pre"])
        r, y, stats = gdn().gdn_resnorm_fwd(x, h, *p, act="silu")
        d = gdn().gdn_resnorm_bwd(x, h, stats, dy, dr, *p, act="silu")
        return {"r": r, "y": y, "stats": stats, "dx": d["dx"], "dh": d["dh"], "dz": d["dz"]}

    whole = run(slice(None))
    for b in range(B):
        for n, x in run(slice(b, b + 1)).items():
            if n == "dz" and gate is None:
                assert x is None
            elif n == "dz" and gate == "sequence":
                assert R.rel(x[0], whole[n][b].double()) <= (2 ** -8 if dt is BF16 else 16 * 2 ** -24)
            else:
                assert torch.equal(x[0], whole[n][b]), n


@pytest.mark.parametrize("carried", [True, False])
@pytest.mark.parametrize("g", [1.0, 2 ** (-2.9 / 128), 2 ** (-3.1 / 128), 2 ** (-11.9 / 128), 2 ** (-12.1 / 128), 2 ** (-11.9 / 384), 2 ** (-12.1 / 384)])
@pytest.mark.parametrize("T", [512, 450])
def test_states_where_the_number_of_terms_changes(T, g, carried):
    """S_T and dS0 in chunks at decays with a chunk's weight on either side of 1/8 and of 2^-12, and without a decay,
    against float64. The weights' powers are off by 4 ulp at most, 2^-21; the tensor cores cut a sum off at each of a
    chunk's eight products, half of 2^-23 of a running sum that grows by its square root, 0.67 x 2^-21 together; the two-term
    chunks' part is less than 2^-22: 2^-20 of the norm. With one term fewer in the last chunk it would be 2^-18, in an earlier
    one 2^-14."""
    a = linattn_inputs(T, 2, T, 2, 4, 64, 72, BF16, g)
    got = linattn(a, state=carried)
    leaves = {n: a[n].double() for n in ("q", "k", "v")}
    leaves["S0"] = a["S0"].double() if carried else torch.zeros_like(a["S0"], dtype=torch.float64)
    (_, S), grads = R.with_grads(lambda **kw: K.linattn(**kw, g=a["g"].double(), lens=None), leaves, (a["dy"].double(), a["dS_T"].double() if carried else None))
    for mine, ref in ((got["S_T"], S), (got["dS0"], grads["S0"])):
        assert R.rel(mine, ref) <= 2 ** -20, R.rel(mine, ref)


def test_states_behind_steps_of_zeros():
    """A row whose last 400 steps add nothing: element by element within 2^-19 of what its steps add before their decay,
    and 2^-20 of itself."""
    a = linattn_inputs(7, 2, 900, 1, 4, 64, 64, BF16)
    a["v"][:, 500:] = 0.0
    _, S = gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"])
    _, ref = K.linattn(a["q"].double(), a["k"].double(), a["v"].double(), a["g"].double(), None, None)
    k = a["k"].double().abs().repeat_interleave(4, 2)
    bound = 2 ** -19 * torch.einsum("bthv,bthk->bhvk", a["v"].double().abs(), k) + 2 ** -20 * ref.abs()
    assert torch.all((S.double() - ref).abs() <= bound)


@pytest.mark.parametrize("dt,T,bad", [(BF16, 500, 200), (BF16, 1600, 900), (BF16, 7, 3), (F32, 500, 200), (F32, 1600, 900)])
def test_what_is_not_finite_reaches(dt, T, bad):
    """A NaN in k and an infinity in v at one step: y and dq of earlier chunks (step by step: of earlier steps), dk and
    dv of later ones, the other head and the other row keep their bits."""
    a = linattn_inputs(5, 2, T, 2, 2, 64, 64, dt)
    clean = linattn(a)
    a["k"][1, bad, 0, 5], a["v"][1, bad, 0, 7] = float("nan"), float("inf")
    dirty = linattn(a)
    unit = 128 if dt is BF16 and T >= 8 else 1
    first, last = bad // unit * unit, (bad // unit + 1) * unit
    for n, x in dirty.items():
        assert torch.equal(x[0], clean[n][0]), n
        if n in ("S_T", "dS0"):
            assert torch.equal(x[1, 1], clean[n][1, 1])
            continue
        assert torch.equal(x[1, :, 1], clean[n][1, :, 1]), n
        kept = slice(0, first) if n in ("y", "dq") else slice(last, T)
        assert torch.equal(x[1, kept, 0], clean[n][1, kept, 0]), n
    assert dirty["y"][1, bad, 0].isnan().all() and dirty["S_T"][1, 0].isnan().any()


@pytest.mark.parametrize("T", [7, 300])
def test_a_query_that_is_not_finite_reaches_its_own_step(T):
    a = linattn_inputs(6, 1, T, 1, 1, 64, 64, BF16)
    clean = linattn(a, train=False)
    a["q"][0, 5, 0, 0] = float("nan")
    y, S = linattn(a, train=False).values()
    keep = torch.arange(T, device="cuda") != 5
    assert y[0, 5].isnan().all() and torch.equal(y[0, keep], clean["y"][0, keep]) and torch.equal(S, clean["S_T"])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_linattn_tensors_of_more_than_2_to_the_31_elements(dt):
    """v, y, dy, dv and the value heads' float32 dq and dk pass 2^31 elements: the last row's last steps against a call of
    its last 568 steps alone (g = 0.8: what lies 500 steps off counts by 2^-160), as far apart as each is off."""
    B, T, Hk, Hv, D, tail = 2, 35000, 2, 256, 128, 568
    if dt is F32:
        T = 34888                                                       # (whole tiles of 16 steps in the tail as well)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=dt)  # noqa: E731
    q, k, v, dy = rnd(B, T, Hk, D), rnd(B, T, Hk, D), rnd(B, T, Hv, D), rnd(B, T, Hv, D)
    assert v.numel() > 2 ** 31
    g = torch.full((Hv,), 0.8, device="cuda")
    cut = [t[1:, T - tail:].contiguous() for t in (q, k, v, dy)]
    y0, S0 = gdn().gdn_linattn_fwd(*cut[:3], g)
    d0 = gdn().gdn_linattn_bwd(*cut[:3], g, cut[3])
    y, S = gdn().gdn_linattn_fwd(q, k, v, g)
    tol = 3 * 2 ** -8 if dt is BF16 else 8e-6
    assert R.rel(y[1, -64:], y0[0, -64:]) <= tol and R.rel(S[1], S0[0]) <= 2 ** -19
    del y, S
    d = gdn().gdn_linattn_bwd(q, k, v, g, dy, want_dS0=False)
    for n in ("dq", "dk", "dv"):
        assert R.rel(d[n][1, -64:], d0[n][0, -64:]) <= tol, n


def test_resnorm_rows_behind_2_to_the_31_elements():
    """Row by row the same bits as a call of the last rows alone."""
    M, D, tail = 265000, 8192, 100
    a = {n: torch.randn(M, D, device="cuda", dtype=BF16) for n in ("x", "h", "dy", "dr")}
    assert a["x"].numel() > 2 ** 31
    w = torch.rand(D, device="cuda")

    def run(rows):
        x, h, dy, dr = (a[n][rows] for n in ("x", "h", "dy", "dr"))
        r, y, stats = gdn().gdn_resnorm_fwd(x, h, None, w, w, w)
        d = gdn().gdn_resnorm_bwd(x, h, stats, dy, dr, None, w, w, w)
        return [t[-tail:].clone() for t in (r, y, stats, d["dx"], d["dh"])]

    assert all(torch.equal(x, y) for x, y in zip(run(slice(None)), run(slice(M - tail, M))))


def linattn_abi(a, lens, state, strides):
    """Forward and backward as a C program calls them: workspaces of exactly the size asked for, and outputs preset to
    NaN, all with guards behind them."""
    from gated_delta_rule_22_gb300 import layer as Ly
    B, T, Hk, Dk = a["q"].shape
    Hv, Dv = a["v"].shape[2:]
    lib, dt, guards = Ly._library(), a["q"].dtype, []
    shape = ctypes.byref(Ly.GdnLinattnShape(B, T, Hk, Hv, Dk, Dv, 1 if dt is BF16 else 0, *strides))

    def guarded(size, dtype):
        n = 1
        for d in size:
            n *= d
        whole = torch.full((n + 64,), float("nan") if dtype is not torch.uint8 else 0x5a, dtype=dtype, device="cuda")
        guards.append(whole[n:])
        return whole[:n].view(size)

    S0, dS_T = (a["S0"], a["dS_T"]) if state else (None, None)
    out = {"y": guarded(a["v"].shape, dt), "S_T": guarded(a["S0"].shape, F32), "dq": guarded(a["q"].shape, dt), "dk": guarded(a["q"].shape, dt),
           "dv": guarded(a["v"].shape, dt), "dS0": guarded(a["S0"].shape, F32)}
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    need = lib.gdn_linattn_fwd_workspace_bytes(shape), lib.gdn_linattn_bwd_workspace_bytes(shape)
    ws = [guarded((n,), torch.uint8) for n in need]
    ins = [_at(a[n]) for n in ("q", "k", "v", "g")] + [_at(S0), _at(lens)]
    assert lib.gdn_linattn_fwd(shape, *ins, _at(out["y"]), _at(out["S_T"]), _at(ws[0]), need[0], stream) == 0
    assert lib.gdn_linattn_bwd(shape, *ins, _at(a["dy"]), _at(dS_T), *(_at(out[n]) for n in ("dq", "dk", "dv", "dS0")), _at(ws[1]), need[1], stream) == 0
    torch.cuda.synchronize()
    assert gdn().gdn_device_status() == 0
    assert all(torch.all(t == 0x5a) if t.dtype is torch.uint8 else t.isnan().all() for t in guards)
    return out


@pytest.mark.parametrize("seed", range(24))
def test_linattn_in_workspaces_of_the_size_asked_for(seed):
    """Random sizes and strides (each of q, k and v packed, or with a stride that TMA reads, or one that it does not, at
    any address), in both types, with rows of any length and NaN behind them: the definition, and nothing written
    behind an output or a workspace."""
    rng = random.Random(seed)
    dt = BF16 if seed % 3 else F32
    B, Hk, group = rng.randint(1, 3), rng.randint(1, 3), rng.choice([1, 2, 3])
    T, dim = rng.choice([1, 2, 7, 8, 63, 64, 65, 129, 300, 700]), lambda: rng.choice([rng.randint(1, 256), 64, 128, 8 * rng.randint(1, 32)])
    Dk, Dv = dim(), dim()
    a = linattn_inputs(seed, B, T, Hk, Hk * group, Dk, Dv, dt)
    lens = torch.tensor([rng.randint(0, T) for _ in range(B)], device="cuda", dtype=torch.int32) if rng.random() < 0.6 else None
    strides = []
    for n in ("q", "k", "v"):
        width, pad = a[n].shape[2] * a[n].shape[3], rng.choice([0, 8, 16, 1, 3])
        before = rng.choice([0, pad // 2, 1, pad]) if pad else 0
        wide = torch.full((B, T, width + pad), float("nan"), device="cuda", dtype=dt)
        a[n] = wide[..., before:before + width].unflatten(-1, a[n].shape[2:]).copy_(a[n])
        strides.append(width + pad)
    for b, n in enumerate([] if lens is None else lens.tolist()):
        for t in ("q", "k", "v", "dy"):
            a[t][b, n:] = float("nan")
    state = rng.random() < 0.5
    got = linattn_abi(a, lens, state, strides)
    leaves = {n: a[n].double() for n in ("q", "k", "v")}
    leaves["S0"] = a["S0"].double() if state else torch.zeros_like(a["S0"], dtype=torch.float64)
    ok = (torch.arange(T, device="cuda") < (T if lens is None else lens[:, None])).expand(B, T)[:, :, None, None]
    cot = (torch.where(ok, a["dy"].double(), 0.0), a["dS_T"].double() if state else None)
    (y, S), grads = R.with_grads(lambda **kw: K.linattn(**kw, g=a["g"].double(), lens=lens), leaves, cot)
    for n, ref in {"y": y, "S_T": S, **{"d" + n: t for n, t in grads.items()}}.items():
        tol = 2 ** -18 if n in ("S_T", "dS0") else 1.5 * 2 ** -8 if dt is BF16 else 4e-6
        assert R.rel(got[n], ref) <= tol, (n, T, Dk, Dv, strides, R.rel(got[n], ref))

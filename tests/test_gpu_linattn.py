"""Linear attention with a decay on the GPU against its float64 definition: forward, gradients, single
steps, both forms (step by step, in chunks), layouts, lengths and decays at which they can go wrong.

Tolerances (2-norm of the error over that of the output). A bf16 output is off by at most 2^-8 of
itself, 0.43 x 2^-8 in the 2-norm (rounding errors are uniform); in chunks the states and their weighted
inputs are rounded to bf16 on the way, and these terms' errors, of either sign, add as the terms' squares do: at
most 0.43 x 2^-8 sqrt(1 + 1 + 1) together, and twice that, 1.5 x 2^-8, where terms partly cancel. float32 outputs, step by step: n roundings of 2^-24 of a sum's
running value, of either sign, and the dot products' Dk: 2^-24 sqrt(2 n + D), up to some 2e-6 at n = 400.
The float32 states of the chunked form hold 24 bits of k and the decay's powers (4 ulp of powf; step by step 2 ulp of exp2 and log2, times
the exponent): 2^-20 covers ages up to log2 = 8, beyond which nothing counts."""
import random

import pytest

torch = pytest.importorskip("torch")
import block_reference as K  # noqa: E402
import layer_reference as R  # noqa: E402

pytestmark = pytest.mark.gpu
TOL = {torch.float32: 4e-6, torch.bfloat16: 1.5 * 2 ** -8}
TOL_STATE = 2 ** -18
BF16, F32 = torch.bfloat16, torch.float32


def gdn():
    import gated_delta_rule_22_gb300
    return gated_delta_rule_22_gb300


def make(seed, B, T, Hk, Hv, Dk, Dv, dt, decay="mixed", wide=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s, scale=1.0: torch.randn(*s, generator=gen, device="cuda") * scale  # noqa: E731

    def rows(H, D, scale=1.0):
        if not wide:
            return rnd(B, T, H, D, scale=scale).to(dt)
        return rnd(B, T, H * D + wide, scale=scale).to(dt)[..., wide // 2:wide // 2 + H * D].unflatten(-1, (H, D))

    g = {"mixed": torch.exp(-torch.exp2(-8.0 * (torch.arange(Hv, device="cuda") + 0.5) / Hv)),
         "one": torch.ones(Hv, device="cuda"), "zero": torch.zeros(Hv, device="cuda"), "tiny": torch.full((Hv,), 1e-30, device="cuda"),
         "long": torch.full((Hv,), 1 - 2 ** -12, device="cuda")}[decay].float()
    return dict(q=rows(Hk, Dk, Dk ** -0.5), k=rows(Hk, Dk), v=rows(Hv, Dv), g=g, S0=rnd(B, Hv, Dv, Dk), dy=rnd(B, T, Hv, Dv).to(dt),
                dS_T=rnd(B, Hv, Dv, Dk, scale=0.3))


def unaligned(t):
    """t in rows of whole 16 bytes, at an address that is none: what the chunked form does not take."""
    n = t.shape[2] * t.shape[3]
    wide = torch.zeros(*t.shape[:2], n // 8 * 8 + 8, device="cuda", dtype=t.dtype)
    return wide[..., 1:1 + n].unflatten(-1, t.shape[2:]).copy_(t)


def reference(a, lens, state, train):
    leaves = {n: a[n].double() for n in ("q", "k", "v")}
    leaves["S0"] = a["S0"].double() if state else torch.zeros_like(a["S0"], dtype=torch.float64)
    f = lambda q, k, v, S0: K.linattn(q, k, v, a["g"].double(), S0, lens)  # noqa: E731
    if not train:
        return f(**leaves), {}
    ok = (torch.arange(a["q"].shape[1], device="cuda") < (10 ** 9 if lens is None else lens[:, None])).expand(a["q"].shape[:2])
    dy = torch.where(ok[:, :, None, None], a["dy"].double(), 0.0)
    return R.with_grads(f, leaves, (dy, a["dS_T"].double() if state else None))


def check(a, lens=None, state=True, train=True, what=""):
    (y, S), grads = reference(a, lens, state, train)
    S0, dS_T = (a["S0"], a["dS_T"]) if state else (None, None)
    got_y, got_S = gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], S0, lens)
    got = {"y": (got_y, y), "S_T": (got_S, S)}
    if train:
        d = gdn().gdn_linattn_bwd(a["q"], a["k"], a["v"], a["g"], a["dy"], S0, lens, dS_T)
        got.update({n: (d[n], grads[n[1:]]) for n in ("dq", "dk", "dv", "dS0")})
    torch.cuda.synchronize()
    assert gdn().gdn_device_status() == 0
    for n, (mine, ref) in got.items():
        tol = TOL_STATE if n in ("S_T", "dS0") else TOL[a["q"].dtype]
        assert R.rel(mine, ref) <= tol, (what, n, R.rel(mine, ref))
    return got


SHAPES = [  # B, T, Hk, Hv, Dk, Dv
    (2, 300, 2, 4, 75, 33), (1, 200, 1, 1, 130, 129), (2, 140, 1, 2, 1, 7), (1, 100, 1, 1, 255, 9),
    (1, 2, 1, 1, 8, 8), (2, 5, 1, 2, 16, 24), (1, 127, 2, 2, 64, 64), (2, 128, 1, 1, 128, 128), (1, 129, 2, 4, 128, 64),
    (3, 300, 1, 3, 64, 128), (2, 257, 2, 2, 96, 120), (1, 400, 1, 2, 192, 128), (1, 260, 1, 1, 256, 256), (2, 140, 2, 2, 40, 75),
    (1, 33, 1, 1, 1, 1), (1, 150, 1, 5, 250, 3), (1, 70, 1, 1, 3, 250), (2, 130, 1, 4, 136, 200),
]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_gradients(shape, dt):
    check(make(1, *shape, dt))


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("decay", ["one", "zero", "tiny", "long"])
def test_decays(decay, dt):
    check(make(2, 2, 290, 1, 2, 64, 64, dt, decay), what=decay)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(5, 200, 1, 2, 64, 64), (5, 300, 2, 2, 128, 40), (5, 131, 1, 1, 24, 33), (5, 520, 1, 1, 64, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_ragged_rows_with_nan_behind_them(shape, dt):
    a = make(3, *shape, dt)
    T = shape[1]
    lens = torch.tensor([T, 0, 1, T - 1, T // 2], device="cuda", dtype=torch.int32)
    for b, n in enumerate(lens.tolist()):
        for t in ("q", "k", "v", "dy"):
            a[t][b, n:] = float("nan") if b % 2 else float("inf")
    got = check(a, lens)
    for n in ("y", "dq", "dk", "dv"):
        for b, L in enumerate(lens.tolist()):
            assert torch.all(got[n][0][b, L:] == 0), n
    assert torch.equal(got["S_T"][0][1], a["S0"][1]) and torch.equal(got["dS0"][0][1], a["dS_T"][1])
    # lengths outside the row are clamped
    wild = torch.tensor([T + 7, -3, 1, T - 1, T // 2], device="cuda", dtype=torch.int32)
    y, S = gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], a["S0"], wild)
    assert torch.equal(y, got["y"][0]) and torch.equal(S, got["S_T"][0])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_without_states(dt):
    a = make(4, 2, 200, 2, 2, 64, 64, dt)
    check(a, state=False)
    y, S = gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], want_S_T=False)
    assert S is None
    d = gdn().gdn_linattn_bwd(a["q"], a["k"], a["v"], a["g"], a["dy"], want_dS0=False)
    assert d["dS0"] is None


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("wide", [16, 6, 1])
def test_column_slices(wide, dt):
    """q, k and v as slices of wider tensors, at any offset: the same results as from packed ones, within the forms' roundings."""
    a = make(5, 2, 150, 2, 2, 64, 64, dt, wide=wide)
    check(a)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", [(8, 8), (64, 64), (128, 128), (192, 128), (256, 256), (75, 40), (130, 1), (1, 3), (33, 100)])
def test_single_step(Dk, Dv, dt):
    a = make(6, 3, 1, 2, 4, Dk, Dv, dt)
    check(a, train=True)
    check(a, state=False, train=False)
    lens = torch.tensor([1, 0, 5], device="cuda", dtype=torch.int32)
    got = check(a, lens, train=False)
    assert torch.equal(got["S_T"][0][1], a["S0"][1]) and torch.all(got["y"][0][1] == 0)
    S = a["S0"].clone()                                                # in place
    y, out = gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], S, lens, S_T=S)
    assert out is S and torch.equal(S, got["S_T"][0]) and torch.equal(y, got["y"][0])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_a_prompt_and_its_tokens_continue_each_other(dt):
    a = make(7, 2, 270, 1, 2, 64, 64, dt)
    (y, S), _ = reference(a, None, True, False)
    cut = 261
    y0, state = gdn().gdn_linattn_fwd(*(a[n][:, :cut].contiguous() for n in "qkv"), a["g"], a["S0"])
    ys = [y0]
    for t in range(cut, 270):
        yt, state = gdn().gdn_linattn_fwd(*(a[n][:, t:t + 1].contiguous() for n in "qkv"), a["g"], state, S_T=state)
        ys.append(yt)
    assert R.rel(torch.cat(ys, 1), y) <= TOL[dt] and R.rel(state, S) <= TOL_STATE


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 200, 1500])
def test_deterministic_and_captured(T, dt):
    """The same bits again, from a captured graph on new inputs too, with rows behind the outputs left alone."""
    a, b = make(8, 2, T, 1, 2, 64, 64, dt), make(9, 2, T, 1, 2, 64, 64, dt)
    run = lambda s: (*gdn().gdn_linattn_fwd(s["q"], s["k"], s["v"], s["g"], s["S0"]),  # noqa: E731
                     *gdn().gdn_linattn_bwd(s["q"], s["k"], s["v"], s["g"], s["dy"], s["S0"], None, s["dS_T"]).values())
    first, again, other = run(a), run(a), run(b)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    live = {n: t.clone() for n, t in a.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(live)
    for want, src in ((first, a), (other, b), (first, a)):
        for n in live:
            live[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out))


def test_gradients_against_differences():
    """<d, gradient> against the central difference of the float32 forward along d: linear in q, v and S0, so
    exact but for roundings (2^-24 of outputs over the step: 1e-4 of the derivative with a step of 0.05)."""
    a = make(10, 1, 180, 1, 2, 24, 20, F32)
    d = gdn().gdn_linattn_bwd(a["q"], a["k"], a["v"], a["g"], a["dy"], a["S0"], None, a["dS_T"])
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dS0")):
        way = torch.randn_like(a[name])
        loss = []
        for sign in (1, -1):
            m = dict(a)
            m[name] = a[name] + sign * 0.05 * way
            y, S = gdn().gdn_linattn_fwd(m["q"], m["k"], m["v"], m["g"], m["S0"])
            loss.append((y.double() * a["dy"].double()).sum() + (S.double() * a["dS_T"].double()).sum())
        numeric, exact = ((loss[0] - loss[1]) / 0.1).item(), (way.double() * d[grad].double()).sum().item()
        assert abs(numeric - exact) <= 1e-3 * abs(exact) + 1e-3 * (way.norm() * d[grad].norm()).item() / way.numel() ** 0.5, name


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1500, 1, 1, 64, 64), (2, 1029, 1, 2, 136, 64), (1, 2100, 1, 1, 24, 40)], ids=lambda s: "x".join(map(str, s)))
def test_long_rows_of_few_heads(shape, dt):
    """Few heads: the chunked form takes a row in segments."""
    check(make(12, *shape, dt), what="long")


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("decay", ["mixed", "one", "zero"])
def test_segments_of_ragged_rows(decay, dt):
    a = make(13, 4, 1300, 1, 1, 64, 64, dt, decay)
    lens = torch.tensor([1300, 130, 700, 0], device="cuda", dtype=torch.int32)
    for b, n in enumerate(lens.tolist()):
        for t in ("q", "k", "v", "dy"):
            a[t][b, n:] = float("nan")
    got = check(a, lens, what=decay)
    assert all(torch.all(got[n][0][b, L:] == 0) for n in ("y", "dq", "dk", "dv") for b, L in enumerate(lens.tolist()))


@pytest.mark.parametrize("wide", [2, 6, 18])
def test_row_strides_that_are_copied(wide):
    """Rows whose stride is no multiple of 8 elements, with NaN between them and behind the sequences."""
    a = make(18, 3, 200, 2, 4, 64, 40, BF16, wide=wide)
    lens = torch.tensor([200, 67, 0], device="cuda", dtype=torch.int32)
    for b, n in enumerate(lens.tolist()):
        for t in ("q", "k", "v", "dy"):
            a[t][b, n:] = float("nan")
    for t in ("q", "k", "v"):
        base = a[t]._base if a[t]._base is not None else a[t]
        flat = base.view(3, 200, -1)
        flat[..., :wide // 2] = float("nan")
        flat[..., flat.shape[-1] - wide // 2:] = float("nan")
    check(a, lens, what="copied")


def test_the_forms_agree():
    """The same bf16 inputs in chunks, and (from addresses that TMA cannot read) step by step: they differ by the
    chunked form's roundings, and the states by their last bits."""
    a = make(14, 2, 600, 2, 4, 128, 64, BF16, wide=16)
    off = dict(a)
    for n in ("q", "k", "v"):
        off[n] = unaligned(a[n])
    y, S = gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], a["S0"])
    y2, S2 = gdn().gdn_linattn_fwd(off["q"], off["k"], off["v"], off["g"], off["S0"])
    assert R.rel(y, y2) <= TOL[BF16] and R.rel(S, S2) <= TOL_STATE and not torch.equal(y, y2)


def test_both_forms_on_many_shapes():
    """Random sizes, lengths, decays and states, bf16, in chunks against step by step: tail chunks of every length
    among them, rows behind which lies NaN, dims in one and two blocks, and no wait that runs out."""
    rng = random.Random(5)
    for _ in range(120):
        B, Hk, group = rng.randint(1, 4), rng.randint(1, 3), rng.choice([1, 1, 2, 3])
        dim = lambda: rng.choice([64, 128, 192, 256, 8 * rng.randint(1, 32), rng.randint(1, 255)])  # noqa: E731
        T = rng.choice([rng.randint(8, 140), rng.randint(120, 600), rng.randint(600, 1500)])
        a = make(rng.randint(0, 10 ** 6), B, T, Hk, Hk * group, dim(), dim(), BF16, rng.choice(["mixed", "mixed", "one", "long", "tiny"]))
        lens = None if rng.random() < 0.4 else torch.tensor([rng.randint(0, T) for _ in range(B)], device="cuda", dtype=torch.int32)
        for b, n in enumerate([] if lens is None else lens.tolist()):
            for t in ("q", "k", "v", "dy"):
                a[t][b, n:] = float("nan")
        off = dict(a)
        odd = a["q"].shape[-1] % 8 or a["v"].shape[-1] % 8              # (copied, at any address)
        for n in ("q", "k", "v", "dy"):
            off[n] = a[n].float() if odd else unaligned(a[n]) if n != "dy" else a[n]
        S0, dS_T = (a["S0"], a["dS_T"]) if rng.random() < 0.5 else (None, None)
        run = lambda s: dict(zip(("y", "S_T"), gdn().gdn_linattn_fwd(s["q"], s["k"], s["v"], s["g"], S0, lens)),  # noqa: E731
                             **gdn().gdn_linattn_bwd(s["q"], s["k"], s["v"], s["g"], s["dy"], S0, lens, dS_T))
        mine, other = run(a), run(off)
        torch.cuda.synchronize()
        assert gdn().gdn_device_status() == 0
        for n, x in mine.items():
            tol = TOL_STATE if n in ("S_T", "dS0") else 2 ** -8 + TOL[BF16]       # (both round their outputs)
            assert R.rel(x, other[n]) <= tol, (n, a["q"].shape, a["v"].shape, lens, R.rel(x, other[n]))


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own memory, give the bits of calls one by one."""
    sets = [make(15 + i, 2, 1000, 1, 2, 64, 64, BF16) for i in range(2)]
    run = lambda a, s: (*gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], a["S0"], stream=s),  # noqa: E731
                        *gdn().gdn_linattn_bwd(a["q"], a["k"], a["v"], a["g"], a["dy"], a["S0"], None, a["dS_T"], stream=s).values())
    want = [run(a, None) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [run(a, s) for a, s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for w, g in zip(want, got) for x, y in zip(w, g))


def test_another_row_or_head_that_is_not_finite():
    """What is not finite stays in its row and head."""
    a = make(17, 3, 400, 2, 2, 64, 64, BF16)
    run = lambda: (*gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], a["S0"]),  # noqa: E731
                   *gdn().gdn_linattn_bwd(a["q"], a["k"], a["v"], a["g"], a["dy"], a["S0"], None, a["dS_T"]).values())
    clean = run()
    a["v"][1, 200, 1] = float("inf")
    a["q"][1, 250, 1, 3] = float("nan")
    for x, y in zip(clean, run()):
        heads = 1 if x.dim() == 4 and x.shape[1] == 2 else 2            # states [B, H, ...], the rest [B, T, H, ...]
        keep = torch.ones_like(x, dtype=torch.bool)
        keep[1].select(heads - 1, 1)[...] = False
        assert torch.equal(x[keep], y[keep])


def test_under_an_explicit_stream():
    """The call under an explicit stream gives the same bits."""
    a = make(11, 2, 300, 1, 2, 128, 128, BF16)
    y, S = gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], a["S0"])
    d = gdn().gdn_linattn_bwd(a["q"], a["k"], a["v"], a["g"], a["dy"], a["S0"], None, a["dS_T"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, S2 = gdn().gdn_linattn_fwd(a["q"], a["k"], a["v"], a["g"], a["S0"], stream=s)
    d2 = gdn().gdn_linattn_bwd(a["q"], a["k"], a["v"], a["g"], a["dy"], a["S0"], None, a["dS_T"], stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(S, S2) and all(torch.equal(d[n], d2[n]) for n in d)

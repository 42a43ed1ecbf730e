"""Linear attention with a decay and the norms around a block on the GPU: calls of the C ABI that the binding
does not make, and what the header says of one row, one prompt or one input beside the others."""
import ctypes

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

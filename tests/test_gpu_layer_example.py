"""The layers of examples/recurrent_layers.py: the library's operators together, as they are used.

Tolerances, relative 2-norm: the same operators on a split sequence round to bf16 at the same places,
but sums run in other orders, so single elements may round the other way: 5e-3, one bf16 rounding.
Against float64, a layer rounds to bf16 about eight times in a row, each 1.1e-3 of the norm on average:
1e-2 (gradients pass the chain twice: 2e-2)."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import layer_reference as R  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_22_gb300 import binding
    if not os.path.exists(binding.LIB_PATH):
        from gated_delta_rule_22_gb300 import build
        build.build()
    import recurrent_layers
    return recurrent_layers


def _x(*shape, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("name", ["GatedDeltaLayer", "SelectiveScanLayer"])
def test_tokens_continue_a_prompt(ex, name):
    layer = getattr(ex, name)()
    x = _x(3, 70, 512)
    whole, end = layer.forward(x)
    assert R.rel(ex.continued(layer, x, 5), whole) <= 5e-3


def _scan_layer64(layer, x, W_in, taps, W_x, W_dt, A_log, dt_bias, D, W_out, lens):
    p = x @ W_in.t()
    u, _ = R.conv(p[..., :layer.C], taps, None, None, lens, "silu")
    r = u @ W_x.t()
    dt = r[..., :layer.R] @ W_dt.t()
    one = lambda t: t.unflatten(-1, (1, layer.N))  # noqa: E731
    y, _ = R.scan(u, dt, A_log, one(r[..., layer.R:layer.R + layer.N]), one(r[..., layer.R + layer.N:]), D, dt_bias,
                  p[..., layer.C:], None, lens)
    return y @ W_out.t() + x


def test_scan_layer_trains(ex):
    """The selective scan layer's output and gradients, on rows of different lengths, against float64."""
    layer = ex.SelectiveScanLayer(width=128, channels=192, states=16, rank=16)
    x, dy = _x(3, 50, 128, seed=1), _x(3, 50, 128, seed=2)
    lens = torch.tensor([50, 0, 23], dtype=torch.int32, device="cuda")
    y, saved = layer.forward(x, train=True, lens=lens)
    got = layer.backward(saved, dy)
    names = ("W_in", "taps", "W_x", "W_dt", "A_log", "dt_bias", "D", "W_out")
    leaves = {"x": x.double(), **{n: getattr(layer, n).double() for n in names}}
    (y64,), g = R.with_grads(lambda **k: _scan_layer64(layer, lens=lens, **k), leaves, (dy.double(),))
    assert R.rel(y, y64) <= 1e-2
    for n, r in g.items():
        assert R.rel(got["d" + n], r) <= 2e-2, n


def _delta_layer64(layer, x, W_in, tq, tk, tv, A_log, dt_bias, w, W_out):
    B, T, _ = x.shape
    q, k, v, z, a, b = layer._split(x @ W_in.t())
    conv = [R.conv(t, f, None, None, None, "silu")[0] for t, f in ((q, tq), (k, tk), (v, tv))]
    unit = lambda t, w_: R.norm(t, layer.Hk, w_.double(), None, None, "none", 1e-6, False).view(B, T, layer.Hk, layer.Dk)  # noqa: E731
    qn, kn = unit(conv[0], layer.w_q), unit(conv[1], layer.w_k)
    vn = conv[2].view(B, T, layer.Hv, layer.Dv)
    g = torch.exp(-torch.exp(A_log) * torch.nn.functional.softplus(a + dt_bias))
    beta = torch.sigmoid(b)
    rep = layer.Hv // layer.Hk
    S = x.new_zeros(B, layer.Hv, layer.Dv, layer.Dk)
    ys = []
    for t in range(T):
        kt, qt = kn[:, t].repeat_interleave(rep, 1), qn[:, t].repeat_interleave(rep, 1)
        S = g[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (vn[:, t] - (S * kt[:, :, None]).sum(-1))
        S = S + u[..., None] * kt[:, :, None]
        ys.append((S * qt[:, :, None]).sum(-1))
    o = torch.stack(ys, 1).reshape(B, T, layer.nv)
    return R.norm(o, layer.Hv, w, None, z, "silu", 1e-5, False) @ W_out.t() + x


def test_delta_layer_trains(ex):
    """The gated delta layer's output and gradients against float64."""
    layer = ex.GatedDeltaLayer(width=128)
    x, dy = _x(2, 70, 128, seed=3), _x(2, 70, 128, seed=4)
    y, saved = layer.forward(x, train=True)
    got = layer.backward(saved, dy)
    leaves = {"x": x.double(), "W_in": layer.W_in.double(), "tq": layer.taps[0].double(), "tk": layer.taps[1].double(),
              "tv": layer.taps[2].double(), "A_log": layer.A_log.double(), "dt_bias": layer.dt_bias.double(), "w": layer.w.double(),
              "W_out": layer.W_out.double()}
    (y64,), g = R.with_grads(lambda **k: _delta_layer64(layer, **k), leaves, (dy.double(),))
    assert R.rel(y, y64) <= 1e-2
    got.update(zip(("dtq", "dtk", "dtv"), got.pop("dtaps")))
    for n, r in g.items():
        assert R.rel(got["d" + n], r) <= 2e-2, n

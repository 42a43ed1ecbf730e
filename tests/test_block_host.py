"""Linear attention with a decay and the norms around a block without a GPU: the host-side refusals of the
C ABI and of its binding, the size queries, and the float64 definitions that the GPU tests compare against.

Pointers of ABI calls are fake addresses that are never dereferenced: every such call returns an
error from the checks that run before anything is enqueued."""
import ctypes
import os

import pytest

from gated_delta_rule_22_gb300 import binding as B
from gated_delta_rule_22_gb300 import layer as Ly

torch = pytest.importorskip("torch")
import block_reference as K  # noqa: E402
import layer_reference as R  # noqa: E402

INVALID, MISALIGNED, UNSUPPORTED, SMALL = -1, -2, -3, -4
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from gated_delta_rule_22_gb300 import build
        build.build()
    return Ly._library()


def linattn_shape(**kw):
    s = dict(B=2, T=300, Hk=2, Hv=4, Dk=64, Dv=48, dtype=1, ldq=0, ldk=0, ldv=0)
    s.update(kw)
    return Ly.GdnLinattnShape(**s)


def resnorm_shape(**kw):
    s = dict(M=12, D=64, gate_rows=3, act=1, post=1, pre=1, dtype=1, eps=1e-5, ldx=0, ldh=0, ldz=0)
    s.update(kw)
    return Ly.GdnResnormShape(**s)


# as in test_layer_host: "!" required, "~" a strided input, "#" a size in bytes
CALLS = {
    "gdn_linattn_fwd": (linattn_shape, "q!~ k!~ v!~ g! S0 lens y! S_T workspace #workspace"),
    "gdn_linattn_bwd": (linattn_shape, "q!~ k!~ v!~ g! S0 lens dy! dS_T dq! dk! dv! dS0 workspace! #workspace"),
    "gdn_resnorm_fwd": (resnorm_shape, "x!~ h!~ z~ scale w_post w_pre r! y! stats"),
    "gdn_resnorm_bwd": (resnorm_shape, "x!~ h!~ z~ scale w_post w_pre stats! dy! dr dx! dh! dz dscale dw_post dw_pre workspace! #workspace"),
}


def call(lib, name, shape, **over):
    args = []
    for i, word in enumerate(CALLS[name][1].split()):
        plain = word.strip("!~")
        if plain.startswith("#"):
            args.append(over.get(plain, 1 << 40))
        else:
            a = over.get(plain, FAKE + (i << 32))
            args.append(None if a is None else ctypes.c_void_p(a))
    return getattr(lib, name)(ctypes.byref(shape) if shape is not None else None, *args, None)


@pytest.mark.parametrize("name", CALLS)
def test_null_misaligned_and_small_buffers(lib, name):
    make, words = CALLS[name]
    assert call(lib, name, None) == INVALID
    for i, word in enumerate(words.split()):
        plain = word.strip("!~")
        if plain.startswith("#"):
            if name.endswith("_bwd"):
                assert call(lib, name, make(), **{plain: 0}) == SMALL
            continue
        if "!" in word:
            assert call(lib, name, make(), **{plain: None}) == INVALID, plain
        at = FAKE + (i << 32)
        assert call(lib, name, make(), **{plain: at + 1}) == MISALIGNED, plain
        if "~" not in word:
            assert call(lib, name, make(), **{plain: at + 8}) == MISALIGNED, plain


@pytest.mark.parametrize("name", ["gdn_linattn_fwd", "gdn_linattn_bwd"])
def test_linattn_shapes(lib, name):
    for kw in (dict(B=0), dict(T=0), dict(Hk=0), dict(Hv=0), dict(Dk=0), dict(Dv=-1), dict(dtype=2), dict(ldq=-1), dict(ldq=127), dict(ldk=127),
               dict(ldv=191)):
        assert call(lib, name, linattn_shape(**kw)) == INVALID, kw
    for kw in (dict(Hv=5), dict(Hk=3), dict(Dk=257), dict(Dv=257), dict(B=65536), dict(Hk=1, Hv=65536), dict(B=65535, T=65535),
               dict(ldv=1 << 41), dict(T=1 << 30, ldq=1 << 20)):
        assert call(lib, name, linattn_shape(**kw)) == UNSUPPORTED, kw
    assert call(lib, "gdn_linattn_fwd", linattn_shape(), S0=FAKE, S_T=FAKE) == INVALID    # in place, more than one step


def test_linattn_workspace(lib):
    need = lambda **kw: lib.gdn_linattn_bwd_workspace_bytes(ctypes.byref(linattn_shape(**kw)))  # noqa: E731
    assert need(Dk=0) == 0 and need(Hv=5) == 0
    rows = 2 * 300 * 4 * 64 * 4                                                              # dq (dk) by value head
    assert need(dtype=0) >= 2 * rows
    assert need(dtype=0, Hk=4, T=40) == 0 and need(Hk=4, T=2000, Dv=64) > 0                   # (segments' states)
    assert need(Hk=4, Dk=63) > need(Hk=4)                                                    # copies of unaligned rows


@pytest.mark.parametrize("name", ["gdn_resnorm_fwd", "gdn_resnorm_bwd"])
def test_resnorm_shapes(lib, name):
    for kw in (dict(M=0), dict(D=0), dict(gate_rows=-1), dict(gate_rows=5), dict(act=3), dict(dtype=2), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("inf")), dict(eps=float("nan")), dict(ldx=63), dict(ldh=-1), dict(ldz=8), dict(post=0), dict(pre=0)):
        assert call(lib, name, resnorm_shape(**kw)) == INVALID, kw
    for kw in (dict(D=16385), dict(M=2 ** 31 - 2 ** 16 + 1, gate_rows=1), dict(M=1 << 24, gate_rows=1, ldh=1 << 20), dict(ldx=1 << 41)):
        assert call(lib, name, resnorm_shape(**kw)) == UNSUPPORTED, kw
    if name == "gdn_resnorm_fwd":
        assert call(lib, name, resnorm_shape(ldx=128), x=FAKE, r=FAKE) == INVALID          # in place, but not packed
        assert call(lib, name, resnorm_shape(pre=0), w_pre=None) == INVALID                # y without its norm
    else:
        assert call(lib, name, resnorm_shape(), z=None) == INVALID                         # dz without z
        assert call(lib, name, resnorm_shape(pre=0), dy=None, w_pre=None, dw_pre=None, dr=None) == INVALID


def test_resnorm_workspace(lib):
    need = lambda **kw: lib.gdn_resnorm_bwd_workspace_bytes(ctypes.byref(resnorm_shape(**kw)))  # noqa: E731
    assert need(M=0) == 0 and need(D=20000) == 0 and need() > 0


def test_binding_refusals(lib):
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    f32 = torch.float32
    ok = dict(q=t(2, 5, 2, 16), k=t(2, 5, 2, 16), v=t(2, 5, 4, 24), g=t(4, dt=f32))
    with pytest.raises(ValueError, match="CUDA"):
        Ly.gdn_linattn_fwd(**ok)
    with pytest.raises(ValueError, match="CUDA"):
        Ly.gdn_linattn_bwd(**ok, dy=t(2, 5, 4, 24))
    for bad in (dict(k=t(2, 5, 2, 17)), dict(v=t(2, 4, 4, 24)), dict(g=t(3, dt=f32)), dict(S0=t(2, 4, 16, 24, dt=f32)),
                dict(lens=torch.zeros(3, dtype=torch.int32)), dict(y=t(2, 5, 4, 16)), dict(S_T=t(2, 4, 16, 24, dt=f32)),
                dict(q=t(2, 2, 5, 16).transpose(1, 2))):
        with pytest.raises(ValueError):
            Ly.gdn_linattn_fwd(**{**ok, **bad})
    for bad in (dict(g=t(4)), dict(v=t(2, 5, 4, 24, dt=f32)), dict(lens=torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(TypeError):
            Ly.gdn_linattn_fwd(**{**ok, **bad})
    with pytest.raises(TypeError):
        Ly.gdn_linattn_fwd(*(t(2, 5, 2, 16, dt=torch.float16),) * 3, t(2, dt=f32))

    x, stats = t(2, 5, 64), t(2, 5, 2, dt=f32)
    with pytest.raises(ValueError, match="CUDA"):
        Ly.gdn_resnorm_fwd(x, x, t(2, 64))
    for bad in (dict(h=t(2, 5, 63)), dict(z=t(5, 64)), dict(z=t(2, 5, 1)), dict(z=t(2, 5, 64, 1)), dict(scale=t(63, dt=f32)), dict(r=t(10, 64)),
                dict(w_pre=t(64, dt=f32), pre=False), dict(w_post=t(64, dt=f32), post=False), dict(y=x, pre=False), dict(act="relu"),
                dict(stats=t(2, 5, dt=f32))):
        with pytest.raises(ValueError):
            Ly.gdn_resnorm_fwd(**{**dict(x=x, h=x), **bad})
    for bad in (dict(), dict(dr=x), dict(dy=x, dr=x, pre=False), dict(pre=False), dict(dy=t(2, 5, 60)), dict(dy=x, stats=t(10, 2, dt=f32))):
        with pytest.raises(ValueError):
            Ly.gdn_resnorm_bwd(**{**dict(x=x, h=x, stats=stats), **bad})
    with pytest.raises(TypeError):
        Ly.gdn_resnorm_fwd(x, x, scale=t(64))


def test_definitions_against_differences():
    """The references' own gradients (autograd) against central differences."""
    torch.manual_seed(0)
    r = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    lens = torch.tensor([7, 3])
    cases = [
        (lambda q, k, v, S0: K.linattn(q, k, v, torch.tensor([0.9, 0.5]), S0, lens), dict(q=r(2, 7, 1, 3), k=r(2, 7, 1, 3), v=r(2, 7, 2, 4), S0=r(2, 2, 4, 3)),
         (r(2, 7, 2, 4), r(2, 2, 4, 3))),
        (lambda **kw: K.resnorm(**kw, post=True, pre=True, act="silu", eps=1e-5), dict(x=r(2, 3, 5), h=r(2, 3, 5), z=r(2, 5), scale=r(5), w_post=r(5), w_pre=r(5)),
         (r(2, 3, 5), r(2, 3, 5))),
    ]
    for f, leaves, cot in cases:
        _, grads = R.with_grads(f, leaves, cot)
        loss = lambda at: sum((o * c).sum() for o, c in zip(f(**at), cot)).item()  # noqa: E731
        for n, t in leaves.items():
            way = torch.randn_like(t)
            numeric = (loss({**leaves, n: t + 1e-5 * way}) - loss({**leaves, n: t - 1e-5 * way})) / 2e-5
            assert abs(numeric - (grads[n] * way).sum().item()) <= 1e-7 * (1 + abs(numeric)), n


def test_a_reset_and_no_decay_are_what_they_say():
    """g = 0: y_t = (q_t . k_t) v_t; g = 1: the plain cumulative form."""
    torch.manual_seed(1)
    q, k, v = (torch.randn(1, 6, 1, 4, dtype=torch.float64) for _ in range(3))
    y, S = K.linattn(q, k, v, torch.zeros(1), torch.randn(1, 1, 4, 4, dtype=torch.float64), None)
    assert torch.allclose(y, (q * k).sum(-1, keepdim=True) * v) and torch.allclose(S[0, 0], v[0, -1, 0, :, None] * k[0, -1, 0])
    y, _ = K.linattn(q, k, v, torch.ones(1), None, None)
    w = torch.tril(torch.einsum("bihd,bjhd->bhij", q, k))
    assert torch.allclose(y, torch.einsum("bhij,bjhd->bihd", w, v))

"""The layer operators without a GPU: the host-side refusals of the C ABI and of its binding, the
size queries, and the float64 definitions that the GPU tests compare against (their gradients
against central differences).

Pointers of ABI calls are fake addresses that are never dereferenced: every such call returns an
error from the checks that run before anything is enqueued."""
import ctypes
import os

import pytest

from gated_delta_rule_22_gb300 import binding as B
from gated_delta_rule_22_gb300 import layer as Ly

torch = pytest.importorskip("torch")
import layer_reference as R  # noqa: E402

INVALID, MISALIGNED, UNSUPPORTED, SMALL = -1, -2, -3, -4
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from gated_delta_rule_22_gb300 import build
        build.build()
    return Ly._library()


def conv_shape(**kw):
    s = dict(B=2, T=9, C=24, W=4, act=1, dtype=1, ldx=0)
    s.update(kw)
    return Ly.GdnConvShape(**s)


def scan_shape(**kw):
    s = dict(B=2, T=40, C=24, N=8, G=2, dtype=1, ldu=0, lddt=0, ldz=0, ldB=0, ldC=0)
    s.update(kw)
    return Ly.GdnScanShape(**s)


def norm_shape(**kw):
    s = dict(M=5, G=3, D=16, act=1, center=1, dtype=1, eps=1e-5, ldx=0, ldz=0)
    s.update(kw)
    return Ly.GdnNormShape(**s)


def linear_shape(**kw):
    s = dict(M=5, N=24, K=16, act=2, dtype=1, ldx=0, ldw=0, ldres=0)
    s.update(kw)
    return Ly.GdnLinearShape(**s)


# every entry point: shape builder, pointers in order ("!" required, "~" strided input: aligned to its
# element only, "#" a size in bytes that follows a buffer)
CALLS = {
    "gdn_conv_fwd": (conv_shape, "x!~ w! bias s0 lens y! s_T"),
    "gdn_conv_bwd": (conv_shape, "x!~ w! bias s0 lens dy! ds_T dx! dw! dbias ds0 workspace! #workspace"),
    "gdn_scan_fwd": (scan_shape, "u!~ dt!~ A_log! B!~ C!~ D dt_bias z~ h0 lens y! h_T ckpt #ckpt workspace #workspace"),
    "gdn_scan_bwd": (scan_shape, "u!~ dt!~ A_log! B!~ C!~ D dt_bias z~ lens ckpt! #ckpt dy! dh_T du! ddt! dA_log! dB! dC! dD "
                                 "ddt_bias dz dh0 workspace! #workspace"),
    "gdn_norm_fwd": (norm_shape, "x!~ w b z~ y! stats"),
    "gdn_norm_bwd": (norm_shape, "x!~ w b z~ stats! dy! dx! dw db dz workspace! #workspace"),
    "gdn_linear_fwd": (linear_shape, "x!~ W!~ bias res~ y! pre workspace #workspace"),
    "gdn_linear_bwd": (linear_shape, "x!~ W!~ pre! dy! dx dW dbias workspace! #workspace"),
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
def test_null_and_misaligned_pointers(lib, name):
    make, words = CALLS[name]
    assert call(lib, name, None) == INVALID
    for word in words.split():
        plain = word.strip("!~")
        if plain.startswith("#"):
            # (the forwards whose small shapes need no workspace would pass this check)
            if plain == "#ckpt" or name.endswith("_bwd"):
                assert call(lib, name, make(), **{plain: 0}) == SMALL, (name, plain)
            continue
        if "!" in word:
            assert call(lib, name, make(), **{plain: None}) == INVALID, (name, plain)
        off = 1 if "~" in word else 8
        assert call(lib, name, make(), **{plain: FAKE + off}) == MISALIGNED, (name, plain)


BAD = [
    ("gdn_conv_fwd", conv_shape, [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(C=-1), INVALID), (dict(W=0), INVALID),
                                  (dict(W=5), UNSUPPORTED), (dict(act=2), INVALID), (dict(act=7), INVALID),
                                  (dict(dtype=3), INVALID), (dict(ldx=23), INVALID), (dict(ldx=-24), INVALID),
                                  (dict(B=70000), UNSUPPORTED), (dict(B=65535, T=65535, C=4096), UNSUPPORTED)]),
    ("gdn_scan_fwd", scan_shape, [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(N=0), INVALID), (dict(G=0), INVALID),
                                  (dict(N=65), UNSUPPORTED), (dict(G=5), UNSUPPORTED), (dict(dtype=-1), INVALID),
                                  (dict(ldu=8), INVALID), (dict(ldB=15), INVALID), (dict(ldz=-1), INVALID),
                                  (dict(B=65535, T=65535), UNSUPPORTED)]),
    ("gdn_norm_fwd", norm_shape, [(dict(M=0), INVALID), (dict(G=0), INVALID), (dict(D=0), INVALID), (dict(act=3), INVALID),
                                  (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
                                  (dict(eps=float("inf")), INVALID), (dict(D=70000), UNSUPPORTED), (dict(ldx=47), INVALID),
                                  (dict(G=65536), UNSUPPORTED)]),
    ("gdn_linear_fwd", linear_shape, [(dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(act=-1), INVALID),
                                      (dict(dtype=2), INVALID), (dict(ldx=15), INVALID), (dict(ldres=23), INVALID),
                                      (dict(M=1 << 24, K=1 << 20), UNSUPPORTED)]),
]


@pytest.mark.parametrize("name,kw,code", [(n, kw, c) for n, _, rows in BAD for kw, c in rows])
def test_bad_shapes(lib, name, kw, code):
    make = CALLS[name][0]
    assert call(lib, name, make(**kw)) == code
    assert call(lib, name.replace("_fwd", "_bwd"), make(**kw)) == code
    size = getattr(lib, name.replace("_fwd", "_bwd_workspace_bytes"))
    assert size(ctypes.byref(make(**kw))) == 0


def test_buffers_too_small_and_aliases(lib):
    s = conv_shape()
    need = lib.gdn_conv_bwd_workspace_bytes(ctypes.byref(s))
    assert need > 0 and call(lib, "gdn_conv_bwd", s, **{"#workspace": need - 1}) == SMALL
    s = scan_shape()
    ck, ws = lib.gdn_scan_ckpt_bytes(ctypes.byref(s)), lib.gdn_scan_bwd_workspace_bytes(ctypes.byref(s))
    assert ck == 2 * 3 * 24 * 8 * 4
    assert call(lib, "gdn_scan_fwd", s, **{"#ckpt": ck - 1}) == SMALL
    assert call(lib, "gdn_scan_bwd", s, **{"#ckpt": ck - 1}) == SMALL
    assert call(lib, "gdn_scan_bwd", s, **{"#workspace": ws - 1}) == SMALL
    long = scan_shape(T=4096)                       # few channels, many steps: the split needs scratch
    need = lib.gdn_scan_fwd_workspace_bytes(ctypes.byref(long))
    assert need > 0 and call(lib, "gdn_scan_fwd", long, **{"#workspace": need - 1}) == SMALL
    assert call(lib, "gdn_scan_fwd", long, workspace=None) == INVALID
    for name, s in (("gdn_norm_bwd", norm_shape()), ("gdn_linear_bwd", linear_shape())):
        need = getattr(lib, name + "_workspace_bytes")(ctypes.byref(s))
        assert need > 0 and call(lib, name, s, **{"#workspace": need - 1}) == SMALL
    # the state in place only for a single step
    assert call(lib, "gdn_conv_fwd", conv_shape(), s0=FAKE, s_T=FAKE) == INVALID
    assert call(lib, "gdn_scan_fwd", scan_shape(), h0=FAKE, h_T=FAKE) == INVALID
    # a gate's gradient without a gate
    assert call(lib, "gdn_scan_bwd", scan_shape(), z=None) == INVALID
    assert call(lib, "gdn_norm_bwd", norm_shape(), z=None) == INVALID


def test_binding_refuses_before_the_library(lib):
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        Ly.gdn_conv_fwd(x, w)
    with pytest.raises(ValueError, match="act"):
        Ly.gdn_conv_fwd(x, w, act="tanh")
    with pytest.raises(ValueError, match="w has shape"):
        Ly.gdn_conv_fwd(x, torch.zeros(7, 4))
    with pytest.raises(TypeError, match="w has dtype"):
        Ly.gdn_conv_fwd(x, w.double())
    with pytest.raises(TypeError, match="lens"):
        Ly.gdn_conv_fwd(x, w, lens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous"):
        Ly.gdn_conv_fwd(torch.zeros(2, 8, 5).transpose(1, 2), w)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        Ly.gdn_conv_fwd(x.half(), w)
    with pytest.raises(ValueError, match="groups"):
        Ly.gdn_norm_fwd(x, 3)
    with pytest.raises(ValueError, match="pre is needed"):
        Ly.gdn_linear_bwd(x, torch.zeros(6, 8), torch.zeros(2, 5, 6), act="silu")
    with pytest.raises(ValueError, match="dy has shape"):
        Ly.gdn_linear_bwd(x, torch.zeros(6, 8), torch.zeros(2, 5, 7))


def test_row_strides_of_slices():
    wide = torch.zeros(3, 5, 40)
    dev = wide.device
    rows = lambda t, inner=1: Ly._rows("t", t, t.shape, torch.float32, dev, inner)  # noqa: E731
    assert rows(wide) == 0
    assert rows(wide[..., 4:20]) == 40
    assert rows(wide[:, :1, 4:20]) == 200            # one step per row: the rows are 5 * 40 apart
    assert rows(wide[:1, :, :16]) == 40
    assert rows(wide[:1, :1, :16]) == 0              # one row in all
    assert rows(wide[..., :24].unflatten(2, (2, 12)), 2) == 40
    for bad in (wide[:, ::2, :16], wide[..., ::2], wide.transpose(0, 1)[..., :16], wide[..., :24].unflatten(2, (12, 2)).transpose(2, 3)):
        with pytest.raises(ValueError, match="contiguous"):
            rows(bad, 2 if bad.dim() == 4 else 1)


def _gradcheck(f, *leaves):
    leaves = [t.clone().requires_grad_(True) for t in leaves]
    assert torch.autograd.gradcheck(f, leaves, eps=1e-6, atol=1e-6)


def test_definitions_against_differences():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    lens = torch.tensor([3, 0], dtype=torch.int32)
    _gradcheck(lambda x, w, b, s: R.conv(x, w, b, s, lens, "silu"), r(2, 4, 3), r(3, 4), r(3), r(2, 3, 3))
    _gradcheck(lambda u, dt, A, B_, C_, D, bias, z, h: R.scan(u, dt, A, B_, C_, D, bias, z, h, lens), r(2, 4, 4), r(2, 4, 4),
               r(4, 3), r(2, 4, 2, 3), r(2, 4, 2, 3), r(4), r(4), r(2, 4, 4), r(2, 4, 3))
    for center in (True, False):
        _gradcheck(lambda x, w, b, z: R.norm(x, 2, w, b, z, "gelu", 1e-5, center), r(3, 8), r(8), r(8), r(3, 8))
    _gradcheck(lambda x, W, b, s: R.linear(x, W, b, s, "gelu"), r(3, 4), r(5, 4), r(5), r(3, 5))

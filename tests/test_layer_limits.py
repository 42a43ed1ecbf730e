"""Sizes at the limits of the layer operators, without a GPU: tensors are shapes alone (device
"meta"), pointers of ABI calls are fake addresses that are never dereferenced."""
import ctypes
import os

import pytest

from gated_delta_rule_22_gb300 import binding as B
from gated_delta_rule_22_gb300 import layer as Ly

torch = pytest.importorskip("torch")
from test_layer_host import call, conv_shape, linear_shape, norm_shape, scan_shape  # noqa: E402

UNSUPPORTED = -3
LONG = 2 ** 32 + 5


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from gated_delta_rule_22_gb300 import build
        build.build()
    return Ly._library()


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("name,make", [
    ("conv", lambda: Ly.gdn_conv_fwd(meta(1, LONG, 1), meta(1, 4, dtype=torch.float32))),
    ("conv", lambda: Ly.gdn_conv_bwd(meta(LONG, 1, 1), meta(1, 4, dtype=torch.float32), meta(LONG, 1, 1))),
    ("scan", lambda: Ly.gdn_scan_fwd(meta(1, LONG, 1), meta(1, LONG, 1), meta(1, 1, dtype=torch.float32), meta(1, LONG, 1, 1),
                                     meta(1, LONG, 1, 1))),
    ("norm", lambda: Ly.gdn_norm_fwd(meta(LONG, 1), 1)),
    ("norm", lambda: Ly.gdn_norm_fwd(meta(2, LONG // 2 + 1, 1), 1)),
    ("linear", lambda: Ly.gdn_linear_fwd(meta(LONG, 1), meta(4, 1))),
    ("linear", lambda: Ly.gdn_linear_bwd(meta(4, 1), meta(LONG, 1), meta(4, LONG))),
    ("gates", lambda: B.make_shape(1, LONG, 1, 1, 32, 4)),
])
def test_sizes_beyond_32_bits_are_refused_not_cut(lib, name, make):
    with pytest.raises(B.GdnError) as e:
        make()
    assert e.value.code == UNSUPPORTED


MOST = 2 ** 31 - 65537


@pytest.mark.parametrize("name,make,kw", [
    ("gdn_conv", conv_shape, lambda n: dict(B=1, T=n, C=1)),
    ("gdn_scan", scan_shape, lambda n: dict(B=1, T=n, C=1, N=1, G=1)),
    ("gdn_norm", norm_shape, lambda n: dict(M=n, G=1, D=1)),
])
def test_rows_whose_counters_would_overflow(lib, name, make, kw):
    """Counters run past the last row by up to a round: the last 65536 values of an int are not taken."""
    size = getattr(lib, name + "_bwd_workspace_bytes")
    assert size(ctypes.byref(make(**kw(MOST)))) > 0
    for n in (MOST + 1, 2 ** 31 - 1):
        assert size(ctypes.byref(make(**kw(n)))) == 0
        for way in ("_fwd", "_bwd"):
            assert call(lib, name + way, make(**kw(n))) == UNSUPPORTED


def test_linear_alignment(lib):
    """Packed bf16 rows of x and W are 16-byte aligned, except single ones and in forwards of few rows.
    Where a call is taken it stops here at its workspace (pointers are never dereferenced)."""
    off = 0x7F0000000000 + 2
    small = {"#workspace": 0}
    for kw, word, code in ((dict(M=33), "x", -2), (dict(M=33), "W", -2), (dict(M=33, N=1), "W", -4), (dict(M=33, dtype=0), "x", -2),
                           (dict(M=33, dtype=0, N=1), "W", -2)):
        if kw.get("dtype") == 0:                       # 2 bytes off: not aligned to the element type itself
            assert call(lib, "gdn_linear_fwd", linear_shape(**kw), **{word: off}, **small) == code
            assert call(lib, "gdn_linear_fwd", linear_shape(**kw), **{word: off + 2}, **small) == -4
        else:
            assert call(lib, "gdn_linear_fwd", linear_shape(**kw), **{word: off}, **small) == code
    for kw, word, code in ((dict(M=5), "x", -2), (dict(M=5), "W", -2), (dict(M=1), "x", -4), (dict(N=1), "W", -4)):
        assert call(lib, "gdn_linear_bwd", linear_shape(**kw), **{word: off}, **small) == code


@pytest.mark.parametrize("name,make,most,kw", [
    ("gdn_conv", conv_shape, 1 << 22, lambda n: dict(B=1, T=2, C=n)),
    ("gdn_scan", scan_shape, 1 << 22, lambda n: dict(B=1, T=2, C=n, N=1, G=1)),
    ("gdn_norm", norm_shape, 65535, lambda n: dict(M=1, G=n, D=1)),
    ("gdn_norm", norm_shape, 65536, lambda n: dict(M=1, G=1, D=n)),
    ("gdn_linear", linear_shape, 4000000, lambda n: dict(M=n)),
    ("gdn_linear", linear_shape, 4000000, lambda n: dict(N=n)),
    ("gdn_linear", linear_shape, 4000000, lambda n: dict(K=n)),
])
def test_documented_sizes(lib, name, make, most, kw):
    """The limits that the header gives, from both sides."""
    size = getattr(lib, name + "_bwd_workspace_bytes")
    assert size(ctypes.byref(make(**kw(most)))) > 0
    assert call(lib, name + "_bwd", make(**kw(most)), **{"#workspace": 0}) == -4
    for way in ("_fwd", "_bwd"):
        assert call(lib, name + way, make(**kw(most + 1))) == UNSUPPORTED

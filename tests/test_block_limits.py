"""Sizes of workspaces and further refusals of the linear attention and of the norms around a block, through the
C ABI without a GPU. Pointers are fake addresses that are never dereferenced: every call returns an error from
the checks that run before anything is enqueued."""
import ctypes

import pytest

pytest.importorskip("torch")
import test_block_host as H  # noqa: E402
from test_block_host import lib  # noqa: E402,F401


@pytest.mark.parametrize("M,D,gate_rows", [(12, 64, 3), (8192, 64, 2048), (65536, 8, 2), (999, 1030, 333), (40000, 16384, 40000)])
def test_resnorm_workspace_holds_the_call_without_a_gate(lib, M, D, gate_rows):  # noqa: F811
    """z is no part of the shape: the size asked for serves gate_rows with a z, and any gate_rows without one."""
    need = lambda **kw: lib.gdn_resnorm_bwd_workspace_bytes(ctypes.byref(H.resnorm_shape(M=M, D=D, **kw)))  # noqa: E731
    assert need(gate_rows=gate_rows) >= need(gate_rows=1) > 0
    assert H.call(lib, "gdn_resnorm_bwd", H.resnorm_shape(M=M, D=D, gate_rows=gate_rows), z=None, dz=None,
                  **{"#workspace": need(gate_rows=gate_rows) - 1}) == H.SMALL


@pytest.mark.parametrize("what", [dict(B=1, T=4096, Hk=1, Hv=1), dict(Dk=63, Hk=4), dict(ldq=129, Hk=2, Hv=4, T=64), dict(dtype=0, B=1, Hk=1, Hv=1, T=4096),
                                  dict(Dk=256, Dv=256, Hk=4)],
                         ids=["segments", "copies", "odd stride", "segments step by step", "wide keys"])
def test_linattn_forward_refuses_a_small_workspace(lib, what):  # noqa: F811
    """Forward calls that need room: for segments' states, copies of rows, float32 outputs."""
    shape = H.linattn_shape(**what)
    need = lib.gdn_linattn_fwd_workspace_bytes(ctypes.byref(shape))
    assert need > 0
    for room in (0, need - 1):
        assert H.call(lib, "gdn_linattn_fwd", shape, **{"#workspace": room}) == H.SMALL
    assert H.call(lib, "gdn_linattn_fwd", shape, workspace=None) == H.INVALID
    assert H.call(lib, "gdn_linattn_fwd", shape, workspace=H.FAKE + 8) == H.MISALIGNED


@pytest.mark.parametrize("what", [dict(T=1), dict(T=7, Hk=4, dtype=0), dict(B=40, Hk=4, T=300)])
def test_linattn_forward_without_a_workspace(lib, what):  # noqa: F811
    assert lib.gdn_linattn_fwd_workspace_bytes(ctypes.byref(H.linattn_shape(**what))) == 0

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

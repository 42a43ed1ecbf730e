"""Calls on an explicit stream, without a GPU: the library, the streams and the allocator are
stand-ins that record under which stream memory was asked for and on which the kernels would run."""
import contextlib

import pytest

from gated_delta_rule_22_gb300 import binding as B
from gated_delta_rule_22_gb300 import layer as Ly

torch = pytest.importorskip("torch")


class Stream:
    device = torch.device("cpu")

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def world(monkeypatch):
    """(side stream, allocations' streams, launches' stream handles)"""
    now, allocs, launches = [Stream(0)], [], []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return lambda *a: 4096

            def launch(*args):
                last = args[-1]
                launches.append(getattr(last, "value", last) or 0)
                return 0
            return launch

    @contextlib.contextmanager
    def under(stream):
        now.append(stream)
        yield
        now.pop()

    def recorded(f):
        def call(*a, **k):
            allocs.append(now[-1].cuda_stream)
            return f(*a, **k)
        return call

    lib = Library()
    for module in (B, Ly):
        monkeypatch.setattr(module, "_require_cuda", lambda t: None)
        monkeypatch.setattr(module, "load_library", lambda *a: lib)
    monkeypatch.setattr(Ly, "_library", lambda: lib)
    monkeypatch.setattr(Ly, "_stream_of", lambda *a: now[-1].cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "stream", under)
    for name in ("empty", "empty_like"):
        f = recorded(getattr(torch, name))
        monkeypatch.setattr(torch, name, f)
        monkeypatch.setattr(Ly, "_" + name, f)
    return Stream(7), allocs, launches


x, w = torch.zeros(2, 40, 24), torch.zeros(24, 4)
bc, A_log = torch.zeros(2, 40, 1, 8), torch.zeros(24, 8)
q, v, g = torch.zeros(1, 64, 2, 32), torch.zeros(1, 64, 2, 4), torch.zeros(1, 64, 2)
saved, vec = torch.zeros(1, 2, 1, 4, 32 * 100), torch.zeros(2)
buf = torch.zeros(1 << 16, dtype=torch.uint8)
CALLS = {
    "conv_fwd": lambda s: Ly.gdn_conv_fwd(x, w, stream=s),
    "conv_bwd": lambda s: Ly.gdn_conv_bwd(x, w, x, stream=s),
    "scan_fwd": lambda s: Ly.gdn_scan_fwd(x, x, A_log, bc, bc, want_ckpt=True, stream=s),
    "scan_bwd": lambda s: Ly.gdn_scan_bwd(x, x, A_log, bc, bc, torch.zeros(2, 3, 24, 8), x, stream=s),
    "norm_fwd": lambda s: Ly.gdn_norm_fwd(x, 3, stream=s),
    "norm_bwd": lambda s: Ly.gdn_norm_bwd(x, 3, torch.zeros(2, 40, 3, 2), x, stream=s),
    "linear_fwd": lambda s: Ly.gdn_linear_fwd(x, torch.zeros(8, 24), stream=s),
    "linear_bwd": lambda s: Ly.gdn_linear_bwd(x, torch.zeros(8, 24), torch.zeros(2, 40, 8), stream=s),
    "fwd": lambda s: B.gdn_fwd(q, q, v, g, g, stream=s),
    "bwd": lambda s: B.gdn_bwd(q, q, v, g, g, torch.zeros(1 << 16)[:256].view(1, 2, 1, 4, 32), v, stream=s),
    "fwd_infer": lambda s: B.gdn_fwd_infer(q, q, v, g, g, stream=s),
    "fwd_rc": lambda s: B.gdn_fwd_rc(q, q, v, g, g, stream=s),
    "bwd_rc": lambda s: B.gdn_bwd_rc(q, q, v, g, g, saved, v, stream=s),
    "fwd_seg": lambda s: B.gdn_fwd_seg(q, q, v, g, g, stream=s),
    "bwd_seg": lambda s: B.gdn_bwd_seg(q, q, v, g, g, buf, v, stream=s),
    "gates_fwd": lambda s: B.gdn_gates_fwd(g, g, vec, vec, stream=s),
    "gates_bwd": lambda s: B.gdn_gates_bwd(g, g, vec, vec, g, g, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_an_explicit_stream(world, name):
    """Scratch and outputs of a call on a stream that is not current are that stream's memory."""
    side, allocs, launches = world
    CALLS[name](side)
    assert allocs and set(allocs) == {7}, allocs
    assert launches == [7]
    allocs.clear()
    launches.clear()
    CALLS[name](None)
    assert allocs and set(allocs) == {0} and launches == [0]


def test_tensors_of_a_device_that_is_not_current(monkeypatch):
    """The library launches on the current device: other devices' tensors are refused before that."""
    other = torch.device("cuda", 1)
    monkeypatch.setattr(Ly, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream(0))
    monkeypatch.setattr(Ly, "_raw_stream", lambda index: 0)
    for stream in (B._stream, Ly._stream_of):
        with pytest.raises(ValueError, match="current device"):
            stream(other)
    assert B._stream(torch.device("cuda", 0)).value in (0, None) and Ly._stream_of(torch.device("cuda", 0)) == 0

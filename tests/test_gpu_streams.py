"""Calls on an explicit stream that is not the current one: the bits of the same calls on the current
stream, while the current stream allocates and overwrites memory right behind each call."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from test_gpu_layer import SCAN, Draw, conv_inputs, gdn, scan_inputs  # noqa: E402,F401


def _calls(gdn):
    """[(name, call)]: each call takes stream= and returns its outputs; inputs are made here."""
    t, lens, dy, ds_T, _ = conv_inputs((3, 130, 264, 4, "bf16", 0, 0, True, [130, 0, 7], "silu"))
    calls = [("conv_fwd", lambda **k: gdn.gdn_conv_fwd(t["x"], t["w"], t["bias"], t["s0"], lens, **k)),
             ("conv_bwd", lambda **k: gdn.gdn_conv_bwd(t["x"], t["w"], dy, t["bias"], t["s0"], lens, ds_T, **k))]
    for case in (SCAN[7], SCAN[13]):
        sc, n, dsy, dh_T = scan_inputs(case)
        args = [sc[k] for k in ("u", "dt", "A_log", "B", "C", "D", "dt_bias", "z")]
        ckpt = gdn.gdn_scan_fwd(*args, sc["h0"], n, want_ckpt=True)[2]
        calls += [("scan_fwd", lambda a=args, h=sc["h0"], n=n, **k: gdn.gdn_scan_fwd(*a, h, n, want_ckpt=True, **k)),
                  ("scan_bwd", lambda a=args, c=ckpt, g=dsy, n=n, d=dh_T, **k: gdn.gdn_scan_bwd(*a[:5], c, g, *a[5:], n, d, **k))]
    r = Draw(4, "bf16")
    x, z, dn, w = r.normal(500, 384), r.normal(500, 384), r.normal(500, 384), r.normal(384, dtype=torch.float32)
    stats = gdn.gdn_norm_fwd(x, 3, w, None, z)[1]
    calls += [("norm_fwd", lambda **k: gdn.gdn_norm_fwd(x, 3, w, None, z, **k)),
              ("norm_bwd", lambda **k: gdn.gdn_norm_bwd(x, 3, stats, dn, w, None, z, **k))]
    for dtype in ("bf16", "f32"):
        r = Draw(5, dtype)
        a, W, dl = r.normal(300, 200), r.normal(264, 200), r.normal(300, 264)
        pre = gdn.gdn_linear_fwd(a, W, act="silu", want_pre=True)[1]
        calls += [("linear_fwd", lambda a=a, W=W, **k: gdn.gdn_linear_fwd(a, W, act="silu", want_pre=True, **k)),
                  ("linear_bwd", lambda a=a, W=W, d=dl, p=pre, **k: gdn.gdn_linear_bwd(a, W, d, p, act="silu", **k))]
    r = Draw(6, "bf16")
    q, k4, v = (torch.nn.functional.normalize(r.normal(2, 192, 2, 64).float(), dim=-1).bfloat16() for _ in range(3))
    g, beta = -torch.rand(2, 192, 2, device="cuda").bfloat16(), torch.rand(2, 192, 2, device="cuda").bfloat16()
    ck = gdn.gdn_fwd(q, k4, v, g, beta)[2]
    calls += [("fwd", lambda **k: gdn.gdn_fwd(q, k4, v, g, beta, **k)[:2]),
              ("fwd_infer", lambda **k: gdn.gdn_fwd_infer(q, k4, v, g, beta, **k)),
              ("bwd", lambda **k: gdn.gdn_bwd(q, k4, v, g, beta, ck, v, **k))]
    return calls


def _tensors(out):
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


def _same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def test_calls_on_a_stream_that_is_not_current(gdn):  # noqa: F811
    calls = _calls(gdn)
    want = [[t.clone() for t in _tensors(call())] for _, call in calls]
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    side.wait_stream(main)
    got = []
    for _, call in calls:
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)                # a millisecond: the call is still waiting when the next line runs
        got.append(_tensors(call(stream=side)))
        for n in (1 << 8, 1 << 12, 1 << 16, 1 << 20, 1 << 22):
            for _ in range(3):
                torch.full((n,), float("nan"), device="cuda")
        assert torch.cuda.current_stream() == main
    main.wait_stream(side)
    for (name, _), a, b in zip(calls, want, got):
        assert len(a) == len(b) and all(_same(x, y) for x, y in zip(a, b)), name
    # outputs used on the current stream and dropped are not handed to the other stream before that use
    for _, call in calls:
        outs = _tensors(call(stream=side))
        main.wait_stream(side)
        torch.cuda._sleep(2_000_000)
        kept = [t.clone() for t in outs]
        del outs
        call(stream=side)
        main.wait_stream(side)
        got.append(kept)
    for (name, _), a, b in zip(calls, want, got[len(calls):]):
        assert all(_same(x, y) for x, y in zip(a, b)), name

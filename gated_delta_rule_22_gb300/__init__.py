"""Gated delta rule training kernels for NVIDIA GB300 (sm_103a).

The compute lives in libgdn.so, a C-ABI library of hand-written CUDA kernels
(include/gdn.h). This package is its thin Python binding.
"""
from importlib import import_module

from .binding import (  # noqa: F401
    GDN_BF16, GDN_F32, GdnError, GdnShape, gdn_bwd, gdn_bwd_noalloc, gdn_bwd_workspace_bytes,
    gdn_ckpt_bytes, gdn_debug_wait_probe, gdn_device_status, gdn_diag_fma_tflops, gdn_fwd,
    gdn_bwd_seg, gdn_fwd_seg, gdn_gates_bwd, gdn_gates_fwd, gdn_last_error, gdn_seg_ckpt_bytes,
    gdn_seg_workspace_bytes, gdn_seg_choose, gdn_fwd_infer, gdn_infer_workspace_bytes, gdn_bwd_rc, gdn_fwd_rc, gdn_rc_bwd_workspace_bytes, gdn_rc_ckpt_bytes,
    gdn_rc_fwd_workspace_bytes, new_rc_ckpt,
    gdn_strerror, gdn_timing_enable, gdn_timing_read, gdn_version,
    header_functions, load_library, make_shape, new_ckpt,
)
# The layer operators' binding needs torch at import; the rest of the package does not before a call.
_LAYER = (
    "GDN_ACT_GELU", "GDN_ACT_NONE", "GDN_ACT_SILU", "GdnConvShape", "GdnLinattnShape", "GdnLinearShape", "GdnNormShape", "GdnResnormShape",
    "GdnScanShape", "gdn_conv_bwd", "gdn_conv_bwd_workspace_bytes", "gdn_conv_fwd", "gdn_linattn_bwd", "gdn_linattn_bwd_workspace_bytes",
    "gdn_linattn_fwd", "gdn_linattn_fwd_workspace_bytes", "gdn_linear_bwd", "gdn_linear_bwd_workspace_bytes", "gdn_linear_fwd",
    "gdn_linear_fwd_workspace_bytes", "gdn_norm_bwd", "gdn_norm_bwd_workspace_bytes", "gdn_norm_fwd", "gdn_resnorm_bwd",
    "gdn_resnorm_bwd_workspace_bytes", "gdn_resnorm_fwd", "gdn_scan_bwd",
    "gdn_scan_bwd_workspace_bytes", "gdn_scan_ckpt_bytes", "gdn_scan_fwd", "gdn_scan_fwd_workspace_bytes",
)


def __getattr__(name):
    if name != "layer" and name not in _LAYER:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    layer = import_module(".layer", __name__)
    globals().update((n, getattr(layer, n)) for n in _LAYER)
    return globals()[name]


def __dir__():
    return sorted({*globals(), *_LAYER, "layer"})

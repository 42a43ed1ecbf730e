"""The package without torch: importing it, and what of it needs no tensors."""
import subprocess
import sys


def _run(code):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)


def test_import_without_torch():
    r = _run("import sys; sys.modules['torch'] = None\n"
             "import gated_delta_rule_22_gb300 as g\n"
             "from gated_delta_rule_22_gb300 import build\n"
             "assert g.make_shape(1, 2, 1, 1, 32, 4).T == 2 and 'gdn_conv_fwd' in dir(g) and g.header_functions()")
    assert r.returncode == 0, r.stderr


def test_layer_names_load_on_first_use():
    r = _run("import sys\n"
             "import gated_delta_rule_22_gb300 as g\n"
             "assert 'torch' not in sys.modules\n"
             "assert g.layer.gdn_conv_fwd is g.gdn_conv_fwd\n"
             "from gated_delta_rule_22_gb300 import gdn_conv_fwd\n"
             "assert g.gdn_conv_fwd is gdn_conv_fwd is g.layer.gdn_conv_fwd and g.GDN_ACT_SILU == 1\n"
             "assert all(getattr(g, n) is getattr(g.layer, n) for n in g._LAYER)\n"
             "try:\n    g.gdn_no_such_call\nexcept AttributeError:\n    pass\nelse:\n    raise SystemExit(1)")
    assert r.returncode == 0, r.stderr

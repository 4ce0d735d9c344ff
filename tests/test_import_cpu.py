"""What importing the package loads."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_star_import_needs_no_torch():
    r = run("import sys\nsys.modules['torch'] = None\nfrom selective_state_space_27_b200 import *\n"
            "assert callable(scan_fwd) and NormArgs and 'selective_state_space_27_b200.serving' not in sys.modules")
    assert r.returncode == 0, r.stderr


def test_serving_operators_load_on_first_use():
    r = run("import sys, selective_state_space_27_b200 as ms\n"
            "names = ('conv_packed_fwd', 'conv_packed_update', 'ssd_packed_fwd', 'ssd_state_update', 'norm_fwd', 'norm_bwd')\n"
            "assert all(n in dir(ms) for n in names) and 'torch' not in sys.modules\n"
            "from selective_state_space_27_b200 import norm_fwd\n"
            "from selective_state_space_27_b200 import serving\n"
            "assert norm_fwd is serving.norm_fwd and all(getattr(ms, n) is getattr(serving, n) for n in names)")
    assert r.returncode == 0, r.stderr

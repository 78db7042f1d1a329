"""What importing the package brings with it."""
import subprocess
import sys

import selective_scan_ss2d_amd as ss
from tests.conftest import ROOT


def test_the_package_imports_no_torch():
    """torch is imported by the first call, not with the names."""
    for how in ("import selective_scan_ss2d_amd as ss; names = ss.__all__; [getattr(ss, n) for n in names]",
                "from selective_scan_ss2d_amd import *; ss1d_delta_forward, ss2d_norm_forward, ss2d_forward"):
        code = how + "; import sys; sys.exit('torch' in sys.modules)"
        assert subprocess.run([sys.executable, "-c", code], cwd=ROOT).returncode == 0, how


def test_every_name_is_listed():
    assert set(ss.__all__) <= set(dir(ss))

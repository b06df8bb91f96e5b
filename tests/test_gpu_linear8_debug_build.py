"""The 8-bit linear layers' tests under the debug build (QGEMM_DEBUG), whose kernels check the coordinates of their copies and
report a failed check as bit 32 of the device error word, which the tests read."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_linear8_under_the_debug_build():
    from block_scaled_quantized_tcgen05_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, QGEMM_DEBUG="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_w8a8.py", "tests/test_gpu_linear8_layers.py",
                        "tests/test_gpu_row_quant.py", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]

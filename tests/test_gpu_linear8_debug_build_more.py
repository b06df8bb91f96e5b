"""The 8-bit linear layers' tests of rows of every length and alignment, and of products over long K, under the bounds-checking
build, which reports a failed check of a load, a store, a copy or a partial sum's slot as bit 32 of the device error word."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = ["tests/test_gpu_row_quant_short.py", "tests/test_gpu_row_quant_long.py", "tests/test_gpu_row_quant_any.py",
         "tests/test_gpu_row_quant_filled.py", "tests/test_gpu_row_quant_eps.py", "tests/test_gpu_row_quant_infinite.py",
         "tests/test_gpu_row_quant_norm_ties.py", "tests/test_gpu_row_quant_longest.py", "tests/test_gpu_w8a8_exact.py"]
# the error word after the last test of a file that does not read it
READ = """
import sys
import pytest
import block_scaled_quantized_tcgen05_gb300 as q
assert q.qgemm_debug_build()
rc = pytest.main([*sys.argv[1:], "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"])
word = q.qgemm_poll_device_error()
print("word", word)
sys.exit(rc or word)
"""


def test_more_of_the_layers_under_the_debug_build():
    from block_scaled_quantized_tcgen05_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, QGEMM_DEBUG="1")
    tests = [t for t in TESTS if os.path.exists(os.path.join(ROOT, t))]
    r = subprocess.run([sys.executable, "-c", READ, *tests], env=env, cwd=ROOT, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout and "word 0" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]

"""The decode-serving tests of special values, windows, bad last pages, graphs and single rows under the bounds-checking build,
which reports a failed check of an offset, of data or scales, as bit 32 of the device error word they all read."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = ["tests/test_gpu_paged_attention_range.py", "tests/test_gpu_paged_attention_infinite.py",
         "tests/test_gpu_paged_attention_window.py", "tests/test_gpu_kv_bad_tail.py", "tests/test_gpu_kv_graphs.py",
         "tests/test_gpu_kv_single_rows.py"]


def test_more_of_decode_serving_under_the_debug_build():
    from block_scaled_quantized_tcgen05_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, QGEMM_DEBUG="1")
    r = subprocess.run([sys.executable, "-m", "pytest", *TESTS, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"], env=env,
                       cwd=ROOT, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]

"""The decode-serving tests under the debug build (QGEMM_DEBUG), whose kernels check the offsets they form
against the planes' extents and report a failed check as bit 32 of the device error word: every test
reads the word and would see it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = ["tests/test_gpu_rope.py", "tests/test_gpu_kv_pages.py", "tests/test_gpu_paged_attention.py",
         "tests/test_gpu_decode_example.py"]


def test_decode_serving_under_the_debug_build():
    from block_scaled_quantized_tcgen05_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, QGEMM_DEBUG="1")
    r = subprocess.run([sys.executable, "-m", "pytest", *TESTS, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"], env=env,
                       cwd=ROOT, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]
    r = subprocess.run([sys.executable, "-c", "import block_scaled_quantized_tcgen05_gb300 as q; print(q.qgemm_debug_build())"],
                       env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.stdout.strip() == "True", r.stdout + r.stderr

"""The offsets' check of the bounds-checking build, compiled for the CPU: data and scale rows alike, and sums that wrap."""
import ctypes
import os
import random
import subprocess

import pytest

from block_scaled_quantized_tcgen05_gb300 import build as qbuild

SHIM = r"""
#include "kv_index.h"
extern "C" int inside(uint32_t p, uint32_t ps, uint32_t r, uint32_t rs, uint32_t h, uint32_t hs, uint32_t unit, uint32_t bytes,
                      int64_t extent) {
    return kvi::row_inside(p, ps, r, rs, h, hs, unit, bytes, extent);
}
"""


@pytest.fixture(scope="module")
def inside(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv_bounds")
    (d / "shim.cpp").write_text(SHIM)
    csrc = os.path.join(os.path.dirname(qbuild.__file__), "csrc")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-I", csrc, str(d / "shim.cpp"), "-o", str(d / "shim.so")], check=True)
    fn = ctypes.CDLL(str(d / "shim.so")).inside
    fn.argtypes = [ctypes.c_uint32] * 8 + [ctypes.c_int64]
    return lambda *a: bool(fn(*a))


def test_last_rows(inside):
    """A cache of 8 pages x 4 heads x 16 rows: its last row is inside, one more byte, row, head or page is not."""
    for unit, row in ((16, 256), (4, 4), (256, 256)):
        rs = row // unit
        hs, ps = 16 * rs, 64 * rs
        extent = 8 * 64 * row
        assert inside(7, ps, 15, rs, 3, hs, unit, row, extent)
        assert not inside(7, ps, 15, rs, 3, hs, unit, row, extent - 1)
        assert not inside(7, ps, 16, rs, 3, hs, unit, row, extent)
        assert not inside(7, ps, 15, rs, 4, hs, unit, row, extent)
        assert not inside(8, ps, 0, rs, 0, hs, unit, row, extent)
        assert inside(0, ps, 0, rs, 0, hs, unit, row, row)


def test_sums_that_wrap(inside):
    """Offsets of 2^32 units and more come out small in 32 bits; the check sees them as they are."""
    big = 1 << 62
    assert inside(1, 0xFFFFFFFF, 0, 16, 0, 0, 16, 256, big)
    assert not inside(1, 0xFFFFFFFF, 1, 1, 0, 0, 16, 256, big)                 # wraps to 0
    assert not inside(1 << 16, 1 << 16, 0, 0, 0, 0, 16, 256, big)              # likewise
    assert not inside(3, 1 << 30, 15, 1 << 26, 3, 1 << 28, 4, 4, big)          # each fits, the sum does not
    assert not inside(0xFFFFFFFF, 0xFFFFFFFF, 0xFFFFFFFF, 0xFFFFFFFF, 0xFFFFFFFF, 0xFFFFFFFF, 1, 1, big)
    rng = random.Random(1)
    for _ in range(2000):
        p, r, h = (rng.choice([0, 1, rng.randrange(1 << 16)]) for _ in range(3))
        ps, rs, hs = (rng.randrange(1 << rng.randint(1, 32)) for _ in range(3))
        unit, n, extent = 1 << rng.randint(2, 20), rng.choice([4, 64, 256]), rng.randrange(1 << rng.randint(8, 60))
        at = p * ps + r * rs + h * hs
        assert inside(p, ps, r, rs, h, hs, unit, n, extent) == (at < 1 << 32 and at * unit + n <= extent)

"""Every kernel file of the 8-bit linear layers checks the addresses that it forms in the debug build (no GPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_quantized_tcgen05_gb300", "csrc")


@pytest.mark.parametrize("name,checks", [("row_quant.cuh", 6), ("w8a8_decode.cu", 2), ("w8a8_pair.cu", 6)])
def test_checks(name, checks):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert len(re.findall(r"QG_IN_(?:BOUNDS|RANGE)\(", code)) >= checks

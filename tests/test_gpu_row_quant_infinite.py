"""Norms whose outputs pass fp32's range where the products of inputs and weights do not."""
import math

import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


@pytest.mark.parametrize("size", [64, 200, 512, 4096, 4101, 16392, 40000])
@pytest.mark.parametrize("dtype", [F, B])
def test_codes_are_zero(size, dtype):
    """Row 0 is one element, whose norm is the root of `size`, times 3e38; the others stay finite."""
    x = torch.zeros(3, size, dtype=dtype, device="cuda")
    x[0, 5] = 1
    x[0, 6] = 0.25
    x[1], x[2] = 1, -1
    w = torch.full((size,), 3e38, device="cuda")
    y, s = torch.full((3, size), 99, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    q.qgemm_norm_quant(x, w, y, s, eps=1e-6)
    assert s[0] == math.inf and not y[0].any()
    ref.check_int8(y[1:], s[1:], ref.norm(x[1:], None, w, 1e-6)[1], ref.norm_error(size))
    c = torch.zeros(3, 8, dtype=dtype, device="cuda")
    a = torch.zeros(3, -(-size // 16) * 16, dtype=torch.int8, device="cuda")[:, :size]
    a.copy_(y)
    ones = torch.ones(8, -(-size // 16) * 16, dtype=torch.int8, device="cuda")[:, :size]
    q.qgemm_w8a8(a, s, ones, torch.full((8,), 1e-30, device="cuda"), c)
    assert c[0].isnan().all() and not c[1:].isnan().any()

"""Rows that fill some of their block's warps and not the others, whose warps take different bodies of the kernel and meet at its
barriers: many rows, so that each block walks a number of them, each with a sum and a maximum of its own."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

B = torch.bfloat16


@pytest.mark.parametrize("size", [520, 1016, 1032, 1528, 2056, 5112, 8200, 12296, 16376, 16392, 24584, 32760])
def test_many_rows(size):
    tokens = 1500
    g = torch.Generator(device="cuda").manual_seed(size)
    x, r = (torch.randn(tokens, size, generator=g, device="cuda").to(B) for _ in "xr")
    # the largest value of every fifth row in the last warp, of the others anywhere; magnitudes apart
    x[::5, -3] = 40
    x.mul_(torch.exp2((torch.arange(tokens, device="cuda") % 17 - 8.0)[:, None]).to(B))
    y, s = torch.empty(tokens, size, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
    for residual in (None, r):
        q.qgemm_norm_quant(x, None, y, s, residual=residual, eps=1e-6)
        for i in range(0, tokens, 500):
            part = slice(i, i + 500)
            want = ref.norm(x[part], None if residual is None else residual[part], None, 1e-6)[1]
            ref.check_int8(y[part], s[part], want, ref.norm_error(size))
        q.qgemm_act_quant(x, y, s, up=residual)
        for i in range(0, tokens, 500):
            part = slice(i, i + 500)
            ref.check_int8(y[part], s[part], ref.act(x[part], None if residual is None else residual[part], "none"), ref.act_error(x, "none"))
        first = y.clone()
        for _ in range(5):
            q.qgemm_act_quant(x, y, s, up=residual)
            assert torch.equal(y, first)
    assert q.qgemm_poll_device_error() == 0

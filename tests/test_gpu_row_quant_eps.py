"""Norms whose eps counts beside the largest means: eps of up to the end of fp32's range."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

B = torch.bfloat16


def check(x, eps):
    tokens, size = x.shape
    want = ref.norm(x, None, None, eps)[1]
    e = ref.norm_error(size)
    y, s = torch.empty(tokens, size, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
    q.qgemm_norm_quant(x, None, y, s, eps=eps)
    ref.check_int8(y, s, want, e)
    y = torch.empty_like(x)
    q.qgemm_norm_quant(x, None, y, eps=eps)
    ref.check_16(y, want, e)
    if size % 32 == 0:
        y, s = (torch.empty(tokens, n, dtype=torch.uint8, device="cuda") for n in (size, size // 32))
        q.qgemm_norm_quant(x, None, y, s, eps=eps)
        ref.check_e4m3(y, s, want, e)


@pytest.mark.parametrize("size", [64, 200, 512, 4096, 4101, 16392, 40000])
@pytest.mark.parametrize("scale,eps", [(1e17, 1e30), (1e19, 3e38), (3e19, 3e38), (1e20, 1e38), (1e22, 3e38), (1e25, 1e-6)])
def test_beside_large_means(size, scale, eps):
    g = torch.Generator(device="cuda").manual_seed(size)
    x = (torch.randn(5, size, generator=g, device="cuda") * scale).to(B)
    x[1] = (x[1].float() * 1e-20).to(B)          # a row whose sum stays in the range, in the same call
    check(x, eps)


@pytest.mark.parametrize("size", [1, 2, 8])
def test_sum_of_mean_and_eps(size):
    """Mean and eps in the range, their sum past it."""
    x = torch.full((3, size), 1.7e19 if size == 1 else 1.2e19, dtype=B, device="cuda")
    x[1] *= -0.5
    if size == 8:
        x *= 0.5
    check(x, 3.3e38)

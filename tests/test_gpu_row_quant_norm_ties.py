"""Integer codes of norms and of products of two operands where the value lies half-way between two: the even one, as the rounding is
defined."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


def codes(x, w, residual=None):
    y, s = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(x), device="cuda")
    q.qgemm_norm_quant(x, w, y, s, residual=residual, eps=1e-6)
    return y


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("size", [128, 200, 512, 1032, 4096, 4101, 8193, 16392, 20001, 33000])
@pytest.mark.parametrize("dtype", [F, B])
def test_half_way(size, dtype, residual):
    """Halves of a row's largest and the other half-way codes that the type holds, whatever the largest is."""
    tokens = 128
    top = 1 + torch.arange(tokens, device="cuda").double() / 128
    h = torch.zeros(tokens, size, dtype=torch.float64, device="cuda")
    h[:, 0] = top
    for k in range(63):
        v = top * (2 * k + 1) / 254
        h[:, 1 + k] = torch.where(v.to(dtype).double() == v, v, 0)
    h[:, -1] = -top / 2
    x = h.to(dtype)
    assert torch.equal(x.double(), h)
    r = None
    if residual:                                     # h = x + r exactly
        r = x / 2
        x = r.clone()
    y = codes(x, None, r)
    assert torch.equal(y.double(), torch.round(h * 127 / top[:, None]))
    assert (y[:, -1] == -64).all()


@pytest.mark.parametrize("size", [128, 256, 512, 4096, 5111, 5112, 14336, 16392, 33000])
def test_every_code(size):
    """bfloat16 rows and gains, whose products have 16 bits: a code's argument lies at 0 or more than 2^-18 from half-way, and its error in
    the kernel (a rounding at up to 127, 2^-18) does not reach that far.  So the codes are those of the formula, all of them."""
    g = torch.Generator(device="cuda").manual_seed(size)
    tokens = 2 ** 22 // size
    x = torch.randn(tokens, size, generator=g, device="cuda").to(B)
    w = (1 + 0.2 * torch.randn(size, generator=g, device="cuda")).to(B)
    hw = x.double() * w.double()
    assert torch.equal(codes(x, w).double(), torch.round(hw * 127 / hw.abs().amax(1, keepdim=True)))


@pytest.mark.parametrize("size", [128, 512, 4096, 5111, 14336, 20001, 28672, 33000])
def test_every_code_of_a_product(size):
    """The same of two bfloat16 operands without an activation."""
    g = torch.Generator(device="cuda").manual_seed(size)
    tokens = 2 ** 21 // size
    x, up = (torch.randn(tokens, size, generator=g, device="cuda").to(B) for _ in "xu")
    y, s = torch.empty(tokens, size, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
    q.qgemm_act_quant(x, y, s, up=up)
    v = x.double() * up.double()
    assert torch.equal(y.double(), torch.round(v * 127 / v.abs().amax(1, keepdim=True)))

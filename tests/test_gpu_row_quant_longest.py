"""The longest rows, off their alignment: the bytes of a row's first elements, counted in 32 bits, pass them."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q

pytestmark = pytest.mark.gpu

F = torch.float16


@pytest.fixture(autouse=True)
def free():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


# (elements before the row's first since 16 bytes, elements of the row): 2 (size + off) is 2^32
@pytest.mark.parametrize("off,size", [(1, (1 << 31) - 1), (7, (1 << 31) - 7)])
def test_first_elements(off, size):
    def row():
        return torch.zeros(size + off, dtype=F, device="cuda")[off:].view(1, size)

    x = row()
    first = torch.tensor([1, -2, 3, -4, 5, -6, 7, -8], dtype=F, device="cuda")
    x[0, :8] = first
    x[0, -1] = 2
    y, s = torch.full((1, size), 99, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    codes = torch.round(first.double() * (127 / 8)).to(torch.int8)

    def check():
        assert torch.equal(y[0, :8], codes)
        assert y[0, -1] == 32 and not y[0, 8:100].any() and not y[0, -100:-1].any()
        assert abs(s.item() - 8 / 127) <= 8 / 127 * 2.0 ** -22

    q.qgemm_act_quant(x, y, s)
    check()
    # the mean of squares is below 2^-23 of eps: y is x but for a unit of the root's
    q.qgemm_norm_quant(x, None, y.fill_(99), s, eps=1.0)
    check()
    up = row().fill_(1)
    q.qgemm_act_quant(x, y.fill_(99), s, up=up)
    check()
    up.zero_()
    q.qgemm_act_quant(x, up)
    assert torch.equal(up[0, :8], first) and up[0, -1] == 2
    assert q.qgemm_poll_device_error() == 0

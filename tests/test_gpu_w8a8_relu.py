"""What the integer product's ReLU leaves of rows whose scales are not numbers."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q

pytestmark = pytest.mark.gpu

F = torch.float16


def small(rows, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, (rows, k), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)


@pytest.mark.parametrize("bias,accumulate", [(0, 0), (1, 1)])
@pytest.mark.parametrize("m,n,k", [(1, 64, 256), (16, 64, 256), (64, 64, 256), (200, 64, 256), (300, 4096, 512), (5, 64, 0)])
def test_relu_of_rows_that_are_not_numbers(m, n, k, bias, accumulate):
    """max(x, +0) of NaN is 0, as in the library's other products."""
    a, w = small(m, k, 3), small(n, k, 4)
    sa, sw = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
    b = torch.full((n,), -3.0, dtype=F, device="cuda") if bias else None
    sa[0] = float("nan")
    if m > 1:
        a[m - 1] = 0
        sa[m - 1] = float("inf")
    c = torch.ones(m, n, dtype=F, device="cuda")
    q.qgemm_w8a8_ex(a, sa, w, sw, c, bias=b, accumulate=bool(accumulate), relu=True)
    want = a.double() @ w.double().T + (-3 if bias else 0) + (1 if accumulate else 0)
    if k:
        want[0] = want[m - 1] = 0
    assert torch.equal(c, want.clamp(min=0).to(F))

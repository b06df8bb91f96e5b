"""Weight-only int4 products into a slice of a wider buffer: the columns beside it keep their values, whatever N is."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [301, 302, 300, 304])
@pytest.mark.parametrize("m", [5, 130])
def test_columns_beside_the_output(m, n):
    k = 512
    g = torch.Generator(device="cuda").manual_seed(n)
    a = torch.randn(m, k, generator=g, device="cuda").to(torch.float16)
    w = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.int16).to(torch.uint8)
    scales = torch.full((n, 64), 120, dtype=torch.uint8, device="cuda")[:, :k // 32]
    half = torch.full((n, k // 32), 0.125, dtype=torch.float16, device="cuda")
    codes = torch.stack([w & 15, w >> 4], 2).flatten(1).to(torch.int16)
    codes = torch.where(codes > 7, codes - 16, codes).double()
    for scale, run in ((2.0 ** -7, lambda c: q.qgemm_w4a16(a, q.qgemm_create_tensor(q.INT4, w, scales), c)),
                       (0.125, lambda c: q.qgemm_w4a16_f16s(a, w, half, c))):
        room = torch.full((m, 320), 3.0, dtype=torch.float16, device="cuda")
        run(room[:, :n])
        assert torch.all(room[:, n:] == 3.0)
        want = (a.double() @ codes.T) * scale
        size = (a.double().abs() @ codes.abs().T) * scale
        # fp32 sums of 512 exact products, one fp16 rounding
        assert torch.all((room[:, :n].double() - want).abs() <= want.abs() * 2.0 ** -11 + size * 33 * 2.0 ** -23 + 2.0 ** -25)
    assert q.qgemm_poll_device_error() == 0

"""Operands whose elements lie more than 2^31 apart: offsets in 64 bits."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

F = torch.float16


@pytest.fixture(autouse=True)
def free():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_rows():
    tokens, size = 70000, 32768
    x = torch.empty(tokens, size, dtype=F, device="cuda")
    for i in range(0, tokens, 10000):
        x[i:i + 10000].normal_()
    rows = torch.tensor([0, 1, 65535, 65536, 69998, 69999], device="cuda")
    want = x[rows].double()
    y, s = torch.empty(tokens, size, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
    q.qgemm_norm_quant(x, None, y, s, eps=1e-6)
    ref.check_int8(y[rows], s[rows], ref.norm(want, None, None, 1e-6)[1], ref.norm_error(size))
    y8, s8 = y.view(torch.uint8), torch.empty(tokens, size // 32, dtype=torch.uint8, device="cuda")
    q.qgemm_act_quant(x, y8, s8)
    ref.check_e4m3(y8[rows], s8[rows], want, ref.U32)
    q.qgemm_norm_quant(x, None, x, eps=1e-6)
    ref.check_16(x[rows], ref.norm(want, None, None, 1e-6)[1], ref.norm_error(size))


def test_long_row_apart():
    """One row stride past 2^31 elements."""
    size, apart = 40000, (1 << 31) + 8
    room = torch.empty(apart + size, dtype=F, device="cuda")
    x = torch.as_strided(room, (2, size), (apart, 1))
    x.copy_(torch.randn(2, size, device="cuda"))
    y, s = torch.empty(2, size, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    q.qgemm_act_quant(x, y, s)
    ref.check_int8(y, s, x.double(), 2 * ref.U32)


@pytest.mark.parametrize("norm", [False, True])
def test_longest_row(norm):
    """A row whose last elements are the last that 31 bits count."""
    size = (1 << 31) - 1
    x = torch.empty(1, size, dtype=F, device="cuda")
    for i in range(0, size, 1 << 28):
        x[:, i:i + (1 << 28)].normal_().clamp_(-5, 5)
    x[0, -3] = -6.0
    y, s = torch.full((1, size), 99, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    square = 1.0
    if norm:
        q.qgemm_norm_quant(x, None, y, s, eps=1.0)
        square = sum(x[:, i:i + (1 << 26)].double().square().sum().item() for i in range(0, size, 1 << 26)) / size + 1.0
    else:
        q.qgemm_act_quant(x, y, s)
    # the sum: 2^20 additions in a row in each of 512 threads, at most half a step each
    scale = 6.0 / 127 / square ** 0.5
    assert abs(s.item() - scale) <= scale * ((1 << 20) * ref.U32 if norm else 2 * ref.U32)
    for i in (0, 1 << 30, size - 5000):
        code = x[:, i:i + 5000].double() * (127 / 6.0)
        assert (y[:, i:i + 5000].double() - code).abs().max() <= 0.5 + 127 * 8 * ref.U32
        assert i or (y[:, :5000] != 99).any()
    assert q.qgemm_poll_device_error() == 0


def product(m, n, k, rows, columns):
    a, w = torch.empty(m, k, dtype=torch.int8, device="cuda"), torch.empty(n, k, dtype=torch.int8, device="cuda")
    for t in (a, w):
        for i in range(0, t.shape[0], 8192):
            t[i:i + 8192].random_(-127, 128)
    sa, sw = torch.rand(m, device="cuda") * 1e-3, torch.rand(n, device="cuda") * 1e-3
    c = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    q.qgemm_w8a8(a, sa, w, sw, c)
    rows, columns = torch.tensor(rows, device="cuda"), torch.tensor(columns, device="cuda")
    y, size = ref.product(a[rows], sa[rows], w[columns], sw[columns])
    ref.check_product(c[rows][:, columns], y, size, k, k * 127 ** 2)
    assert q.qgemm_poll_device_error() == 0


def test_large_output():
    product(70000, 32768, 64, [0, 1, 65535, 65536, 69999], [0, 5, 32767])


def test_large_tokens():
    """Tokens past 2^31 bytes, in several slices of scratch."""
    product(40000, 256, 65536, [0, 3, 4095, 4096, 32767, 32768, 39999], [0, 255])


@pytest.mark.parametrize("m", [1, 16, 40])
def test_large_weights(m):
    product(m, 40000, 65536, [0, m - 1], [0, 32767, 32768, 39999])

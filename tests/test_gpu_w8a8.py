"""Product of 8-bit integers with token and channel scales on the GPU against exact integer sums."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16


def codes(rows, k, seed, top=127, pad=0):
    """[rows, k] codes in rows padded to 16 bytes (and `pad` more) with bytes that are not to be read as data."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = -(-k // 16) * 16 + pad
    room = torch.randint(-128, 128, (rows, width), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    room[:, :k] = torch.randint(-top - 1, top + 1, (rows, k), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    return room[:, :k]


def scales(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp2(torch.rand(n, generator=g, device="cuda") * 8 - 14)


def run(m, n, k, dtype, bias=False, accumulate=False, relu=False, top=127, pad=0, cpad=0):
    a, w = codes(m, k, 1, top, pad), codes(n, k, 2, top, pad)
    sa, sw = scales(m, 3), scales(n, 4)
    b = torch.randn(n, device="cuda").to(dtype) if bias else None
    room = torch.randn(m + 1, n + cpad, device="cuda").to(dtype)
    c = room[:m, :n]
    old, before = c.clone(), room.clone()
    if accumulate or relu:
        q.qgemm_w8a8_ex(a, sa, w, sw, c, bias=b, accumulate=accumulate, relu=relu)
    else:
        q.qgemm_w8a8(a, sa, w, sw, c, bias=b)
    y, size = ref.product(a, sa, w, sw, b, old if accumulate else None, relu)
    ref.check_product(c, y, size, k, k * (top + 1) ** 2)
    assert torch.equal(room[m], before[m]) and torch.equal(room[:, n:], before[:, n:])
    assert q.qgemm_poll_device_error() == 0


@pytest.mark.parametrize("m", [1, 2, 3, 8, 9, 16, 17, 31, 32, 33, 64, 65, 100, 128, 129, 256, 257, 600])
@pytest.mark.parametrize("n,k", [(256, 512), (1, 16), (37, 130), (264, 1), (1000, 1032), (512, 4096)])
def test_shapes(m, n, k):
    run(m, n, k, F if (m + n) % 2 else B, bias=m % 3 == 0)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("m", [1, 5, 16, 40, 100, 200, 300])
@pytest.mark.parametrize("accumulate,relu,bias", [(1, 0, 0), (0, 1, 1), (1, 1, 1), (0, 0, 1)])
def test_epilogue(m, dtype, accumulate, relu, bias):
    run(m, 333, 784, dtype, bias, accumulate, relu)
    run(m, 384, 2048, dtype, bias, accumulate, relu)


@pytest.mark.parametrize("m", [1, 4, 12, 16, 48, 96, 300])
@pytest.mark.parametrize("n,k", [(4096, 4096), (1024, 14336), (28672, 512), (152, 28672)])
def test_projections(m, n, k):
    run(m, n, k, B)


@pytest.mark.parametrize("m,n,k", [(1024, 2048, 4096), (777, 5003, 4111), (2048, 768, 8192), (4100, 512, 130)])
def test_large(m, n, k):
    run(m, n, k, F, bias=True)


@pytest.mark.parametrize("m", [1, 16, 20, 70, 130, 260])
def test_strides(m):
    run(m, 300, 500, F, pad=48, cpad=0)
    run(m, 301, 500, B, pad=16, cpad=3)
    run(m, 304, 512, B, pad=0, cpad=8)


@pytest.mark.parametrize("m", [1, 7, 16, 40, 130, 300])
def test_exact_sums(m):
    """Codes whose sums stay below 2^24 give the exact integer: outputs equal to those of 64 bits, rounded."""
    a, w = codes(m, 1000, 1, 9), codes(300, 1000, 2, 9)
    one_m, one_n = torch.ones(m, device="cuda"), torch.ones(300, device="cuda")
    c = torch.empty(m, 300, dtype=F, device="cuda")
    q.qgemm_w8a8(a, one_m, w, one_n, c)
    assert torch.equal(c, (a.double() @ w.double().T).to(F))


@pytest.mark.parametrize("m", [1, 16, 64, 200])
@pytest.mark.parametrize("k", [1024, 28672, 140000])
def test_largest_sums(m, k):
    """Every product +-2^14: sums to 2^31 and beyond, past what 32-bit integers hold."""
    n = 40
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    sa, sw = scales(m, 1), scales(n, 2)
    c = torch.empty(m, n, dtype=B, device="cuda")
    q.qgemm_w8a8(a, sa, w, sw, c)
    y, size = ref.product(a, sa, w, sw)
    ref.check_product(c, y, size, k, k * 2 ** 14)


@pytest.mark.parametrize("m", [1, 16, 64, 200])
def test_one_hot(m):
    """Every position of K reaches its product: row n of W is one at k = n."""
    k = 400
    a = codes(m, k, 1)
    w = torch.zeros(k, 400, dtype=torch.int8, device="cuda")
    w[torch.arange(k), torch.arange(k)] = 1
    c = torch.empty(m, k, dtype=F, device="cuda")
    q.qgemm_w8a8(a, torch.ones(m, device="cuda"), w, torch.ones(k, device="cuda"), c)
    assert torch.equal(c, a.to(F))


@pytest.mark.parametrize("m", [1, 16, 64, 200])
def test_scales_that_are_not_numbers(m):
    """A NaN or infinite token scale makes its row NaN or infinite and no other."""
    a, w = codes(m, 256, 1), codes(64, 256, 2)
    sa, sw = scales(m, 3), scales(64, 4)
    sa[0] = float("nan")
    a[m - 1] = 0
    if m > 1:
        sa[m - 1] = float("inf")
    c = torch.empty(m, 64, dtype=F, device="cuda")
    q.qgemm_w8a8(a, sa, w, sw, c)
    assert torch.all(c[0].isnan()) and torch.all(c[m - 1].isnan())
    if m > 2:
        assert torch.all(c[1:m - 1].isfinite())


@pytest.mark.parametrize("bias,accumulate,relu", [(0, 0, 0), (1, 0, 0), (1, 1, 1)])
def test_no_k(bias, accumulate, relu):
    m, n = 5, 70
    a, w = torch.empty(m, 0, dtype=torch.int8, device="cuda"), torch.empty(n, 0, dtype=torch.int8, device="cuda")
    b = torch.randn(n, device="cuda").to(F) if bias else None
    c = torch.randn(m, n, device="cuda").to(F)
    want = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    want += b.double() if bias else 0
    want += c.double() if accumulate else 0
    q.qgemm_w8a8_ex(a, scales(m, 1), w, scales(n, 2), c, bias=b, accumulate=bool(accumulate), relu=bool(relu))
    assert torch.equal(c, (want.clamp(min=0) if relu else want).to(F))


def test_nothing_to_write():
    a, w = codes(3, 32, 1), codes(4, 32, 2)
    q.qgemm_w8a8(a[:0], scales(3, 1)[:0], w, scales(4, 2), torch.empty(0, 4, dtype=F, device="cuda"))
    q.qgemm_w8a8(a, scales(3, 1), w[:0], scales(4, 2)[:0], torch.empty(3, 0, dtype=F, device="cuda"))


@pytest.mark.parametrize("m", [1, 16, 64, 300])
def test_repeatable(m):
    a, w, sa, sw = codes(m, 4096, 1), codes(1024, 4096, 2), scales(m, 3), scales(1024, 4)
    first = None
    for _ in range(4):
        c = torch.empty(m, 1024, dtype=B, device="cuda")
        q.qgemm_w8a8(a, sa, w, sw, c)
        assert first is None or torch.equal(c, first)
        first = c

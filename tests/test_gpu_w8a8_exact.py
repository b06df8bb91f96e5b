"""Products of 8-bit integers over long K, in whole waves, shared tiles and clusters, whose outputs hold every unit of the sums: a product
lost or counted twice shows."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q

pytestmark = pytest.mark.gpu

F = torch.float16


def small(rows, k, seed):
    """Codes of -3 .. 3 in rows padded to 16 bytes: 28672 products have a standard deviation of 677, so that nearly all sums lie
    where a half holds every integer, and all below 2^24."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    room = torch.full((rows, -(-k // 16) * 16), 77, dtype=torch.int8, device="cuda")
    room[:, :k] = torch.randint(-3, 4, (rows, k), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    return room[:, :k]


def check(m, n, k):
    a, w = small(m, k, 1), small(n, k, 2)
    c = torch.empty(m, n, dtype=F, device="cuda")
    q.qgemm_w8a8(a, torch.ones(m, device="cuda"), w, torch.ones(n, device="cuda"), c)
    # exact in 32 bits too: every partial sum is below 2^24, in any order
    want = torch.cat([a[i:i + 1024].double() @ w.double().T for i in range(0, m, 1024)])
    assert float((want.abs() <= 2048).double().mean()) > 0.99
    assert torch.equal(c, want.to(F))
    assert q.qgemm_poll_device_error() == 0


# a weight stream with K over clusters, with K whole, with few blocks of rows
@pytest.mark.parametrize("m", [1, 8, 16])
@pytest.mark.parametrize("n,k", [(152, 28672), (4096, 4096), (28672, 1024), (1000, 28671), (33, 28000), (8192, 8192)])
def test_few_tokens(m, n, k):
    check(m, n, k)


@pytest.mark.parametrize("m,n,k", [(20, 4096, 4096), (32, 152, 28672), (40, 512, 8192), (64, 1536, 2560), (33, 2048, 2047)])
def test_stream_past_16_tokens(m, n, k):
    check(m, n, k)


# tiles of 64, 128 and 256 tokens: one a pair, cut evenly or into equal ranges of K, after whole waves and without any; ragged
@pytest.mark.parametrize("m,n,k", [(64, 1024, 14336), (64, 28672, 2048), (64, 28672, 28672), (50, 5003, 4111), (200, 1000, 4096),
                                   (128, 28672, 8192), (100, 4096, 8192), (200, 2048, 14336), (200, 12288, 4096), (200, 12288, 14336),
                                   (300, 4096, 4096), (777, 5003, 4111), (333, 5003, 28671), (2560, 4096, 4096), (5000, 5000, 1000),
                                   (500, 12288, 14336), (1000, 5003, 8191), (1500, 1000, 14336), (500, 8192, 4096), (512, 19456, 4100)])
def test_pairs(m, n, k):
    check(m, n, k)

"""Rows of 16385 elements and more, many of them: rings that turn (parts of rows for two operands to INT8), rows read twice,
at any alignment, in place, and the special values that take a norm's codes from y itself."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16
# parts that end inside a row's last, a whole ring, past what a block holds
SIZES = [16392, 16389, 28672, 32768, 32771, 53248]


def rows(tokens, size, dtype, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(tokens, size + pad, dtype=dtype, device="cuda")[:, :size]
    x.copy_(torch.randn(tokens, size, generator=g, device="cuda"))
    return x.mul_(torch.exp2((torch.arange(tokens, device="cuda") % 9 - 4.0)[:, None]).to(dtype))


def check(y, s, want, e):
    """By groups of rows: the reference takes 64 bits an element."""
    for i in range(0, len(y), 256):
        if s is None:
            ref.check_16(y[i:i + 256], want(i), e(i))
        elif s.dim() == 1:
            ref.check_int8(y[i:i + 256], s[i:i + 256], want(i), e(i))
        else:
            ref.check_e4m3(y[i:i + 256], s[i:i + 256], want(i), e(i))


@pytest.mark.parametrize("tokens", [2, 153, 700])
@pytest.mark.parametrize("size", SIZES)
def test_gated_to_int8(tokens, size):
    x, up = rows(tokens, size, B, 1, pad=3), rows(tokens, size, B, 2)
    room = torch.full((tokens, size + 5), 99, dtype=torch.int8, device="cuda")
    y, s = room[:, :size], torch.empty(tokens, device="cuda")
    for kind in ("silu", "none"):
        q.qgemm_act_quant(x, y, s, up=up, activation=kind)
        check(y, s, lambda i: ref.act(x[i:i + 256], up[i:i + 256], kind), lambda i: ref.act_error(x[i:i + 256], kind))
    assert (room[:, size:] == 99).all() and q.qgemm_poll_device_error() == 0


@pytest.mark.parametrize("size", SIZES)
def test_norm_to_int8(size):
    tokens = 700
    x, r, w = rows(tokens, size, F, 3), rows(tokens, size, F, 4, pad=8), torch.rand(size, device="cuda") + 0.5
    y, s = torch.empty(tokens, size, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
    q.qgemm_norm_quant(x, w, y, s, residual=r, eps=1e-5)
    check(y, s, lambda i: ref.norm(x[i:i + 256], r[i:i + 256], w, 1e-5)[1], lambda i: ref.norm_error(size))
    assert q.qgemm_poll_device_error() == 0


@pytest.mark.parametrize("size", [32768, 53248, 65568])
def test_blocks_of_32(size):
    tokens = 333
    x, up, w = rows(tokens, size, B, 5), rows(tokens, size, B, 6, pad=1), torch.rand(size, device="cuda") + 0.5
    y, s = (torch.empty(tokens, n, dtype=torch.uint8, device="cuda") for n in (size, size // 32))
    q.qgemm_act_quant(x, y, s, up=up, activation="gelu")
    check(y, s, lambda i: ref.act(x[i:i + 256], up[i:i + 256], "gelu"), lambda i: ref.act_error(x[i:i + 256], "gelu"))
    q.qgemm_norm_quant(x, w, y, s, residual=up, eps=1e-5)
    check(y, s, lambda i: ref.norm(x[i:i + 256], up[i:i + 256], w, 1e-5)[1], lambda i: ref.norm_error(size))


@pytest.mark.parametrize("size", [20001, 32771, 53248])
def test_in_place(size):
    """Rows at any alignment that are their own output, beside the sum that takes the residual's place."""
    tokens = 400
    x, r = rows(tokens, size, B, 7), rows(tokens, size, B, 8)
    x0, r0 = x.clone(), r.clone()
    q.qgemm_norm_quant(x, None, x, residual=r, residual_out=r, eps=1e-5)
    want = [ref.norm(x0[i:i + 256], r0[i:i + 256], None, 1e-5) for i in range(0, tokens, 256)]
    check(x, None, lambda i: want[i // 256][1], lambda i: ref.norm_error(size))
    check(r, None, lambda i: want[i // 256][0], lambda i: ref.U32)
    x.copy_(x0)
    q.qgemm_act_quant(x, x, up=r0, activation="silu")
    check(x, None, lambda i: ref.act(x0[i:i + 256], r0[i:i + 256], "silu"), lambda i: ref.act_error(x0[i:i + 256], "silu"))


@pytest.mark.parametrize("size", [64, 544, 5120, 16392, 40000])
def test_codes_of_a_norm_at_the_ends_of_the_range(size):
    """Weights so small, or sums so large, that h w is subnormal, infinite or below the least scale, where y need not be."""
    tokens = 8
    x = rows(tokens, size, B, 9)
    small, large = torch.exp2(torch.tensor(-120.0)), torch.exp2(torch.tensor(100.0))
    scale = torch.tensor([1.0, small, small ** 1.05, large, 1.2 * large, 0.0, 1.0, small * 0.5], device="cuda")
    x.copy_((x.float() * scale[:, None]).to(B))
    for weight in (1.0, 2.0 ** -20, 2.0 ** -90, 2.0 ** 100):
        w = torch.full((size,), weight, device="cuda")
        y, s = torch.empty(tokens, size, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
        q.qgemm_norm_quant(x, w, y, s, eps=2.0 ** -64)
        ref.check_int8(y, s, ref.norm(x, None, w, 2.0 ** -64)[1], ref.norm_error(size))

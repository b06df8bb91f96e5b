"""Rows of 8193 to 16384 elements at any alignment, with a second operand and without: what one operand off its alignment
sends past the aligned kernels, to each output."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16
TOKENS = 3


def rows(tokens, size, dtype, seed, off=0):
    """Rows whose first element lies `off` elements past 16 bytes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(tokens * (size + 8) + 8, dtype=dtype, device="cuda")[off:off + tokens * (size + 8)].view(tokens, size + 8)[:, :size]
    x.copy_(torch.randn(tokens, size, generator=g, device="cuda"))
    return x


def outputs(tokens, size, to, dtype, off=0):
    def room(t):
        return torch.zeros(tokens * size + off, dtype=t, device="cuda")[off:].view(tokens, size)

    if to == "16":
        return room(dtype), None
    if to == "int8":
        return room(torch.int8), torch.empty(tokens, device="cuda")
    return room(torch.uint8), torch.empty(tokens, size // 32, dtype=torch.uint8, device="cuda")


def check(y, s, want, e):
    if s is None:
        ref.check_16(y, want, e)
    elif s.dim() == 1:
        ref.check_int8(y, s, want, e)
    else:
        ref.check_e4m3(y, s, want, e)


def both(size, to, dtype, second, xoff=0, yoff=0, woff=0, off2=0):
    x, r = rows(TOKENS, size, dtype, size, xoff), rows(TOKENS, size, dtype, size + 1, off2) if second else None
    w = rows(1, size, dtype, size + 2, woff)[0]
    h = torch.empty_like(r) if second else None
    y, s = outputs(TOKENS, size, to, dtype, yoff)
    q.qgemm_norm_quant(x, w, y, s, residual=r, residual_out=h, eps=1e-5)
    wh, wy = ref.norm(x, r, w, 1e-5)
    check(y, s, wy, ref.norm_error(size))
    if second:
        ref.check_16(h, wh, ref.U32)
    for kind in ("none", "silu"):
        y, s = outputs(TOKENS, size, to, dtype, yoff)
        q.qgemm_act_quant(x, y, s, up=r, activation=kind)
        check(y, s, ref.act(x, r, kind), ref.act_error(x, kind))


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("to", ["int8", "e4m3", "16"])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("size", [8192, 8193, 8224, 9217, 9248, 9999, 11265, 11296, 12288, 12289, 16352, 16383, 16384])
def test_sizes(size, dtype, to, second):
    if to == "e4m3" and size % 32:
        pytest.skip("blocks of 32")
    both(size, to, dtype, second, xoff=1)


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("to", ["int8", "e4m3", "16"])
@pytest.mark.parametrize("off", [dict(xoff=1), dict(xoff=7), dict(yoff=1), dict(woff=1), dict(off2=3)])
def test_one_operand_off_its_alignment(off, to, second):
    both(12288, to, F, second, **off)


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("to", ["int8", "16"])
def test_every_block(to, second):
    """A size for each number of warps that a row of the range may take, at either end of it."""
    for size in range(8192, 16385, 512):
        for edge in (-1, 0, 1):
            if size + edge <= 16384:
                both(size + edge, to, B, second, xoff=1)


@pytest.mark.parametrize("size", [9217, 12289])
def test_many_rows(size):
    """Rows beyond a block's first."""
    x = rows(1000, size, B, 1, 1)
    y, s = outputs(1000, size, "int8", B)
    q.qgemm_norm_quant(x, None, y, s, eps=1e-5)
    ref.check_int8(y, s, ref.norm(x, None, None, 1e-5)[1], ref.norm_error(size))
    q.qgemm_act_quant(x, y, s)
    ref.check_int8(y, s, x.double(), 2 * ref.U32)
    assert q.qgemm_poll_device_error() == 0

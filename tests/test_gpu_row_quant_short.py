"""Rows of up to 256 elements (heads), several to a warp: rows that take the special paths beside rows that do not, counts that
leave a warp part of its rows, in place, nothing written beside them."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16
SIZES = [8, 32, 96, 128, 136, 160, 248, 256, 264]


def inputs(tokens, size, dtype, seed, special):
    """`special`: every third row too large for its sum of squares, or too small for its scale, or of zeros."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, size, generator=g, device="cuda")
    if special:
        scale = torch.tensor([1.0, 2.0 ** 100, 1.0, 1.0, 2.0 ** -120, 1.0, 0.0, 1.0], device="cuda")
        x = x * scale[torch.arange(tokens, device="cuda") % 8][:, None]
    return x.to(dtype)


def guarded(tokens, size, dtype, fill):
    room = torch.full((tokens + 2, size + 8), fill, device="cuda").to(dtype)
    return room, room[1:-1, :size]


def beside(room, size, fill):
    same = room == torch.full((), fill, device="cuda").to(room.dtype)
    return bool(same[0].all() and same[-1].all() and same[:, size:].all())


@pytest.mark.parametrize("tokens", [1, 3, 5, 30, 1003])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("special", [False, True])
def test_norm(tokens, size, special):
    dtype = B if special else F
    x, r, w = inputs(tokens, size, dtype, 1, special), inputs(tokens, size, dtype, 2, False), torch.rand(size, device="cuda") + 0.5
    for residual in (None, r):
        h, y = ref.norm(x, residual, w, 1e-5)
        room, out = guarded(tokens, size, torch.int8, 99)
        sums, total = guarded(tokens, size, dtype, 7.0)
        s = torch.empty(tokens + 2, device="cuda").fill_(-5.0)
        q.qgemm_norm_quant(x, w, out, s[1:-1], residual=residual, residual_out=None if residual is None else total, eps=1e-5)
        ref.check_int8(out, s[1:-1], y, ref.norm_error(size))
        assert beside(room, size, 99) and float(s[0]) == -5.0 == float(s[-1])
        if residual is not None:
            ref.check_16(total, h, ref.U32)
            assert beside(sums, size, 7.0)
        room, out = guarded(tokens, size, dtype, 7.0)
        q.qgemm_norm_quant(x, w, out, residual=residual, eps=1e-5)
        ref.check_16(out, y, ref.norm_error(size))
        assert beside(room, size, 7.0)
        if size % 32 == 0:
            (room, out), (rooms, scales) = guarded(tokens, size, torch.uint8, 99), guarded(tokens, size // 32, torch.uint8, 99)
            q.qgemm_norm_quant(x, w, out, scales, residual=residual, eps=1e-5)
            ref.check_e4m3(out, scales, y, ref.norm_error(size))
            assert beside(room, size, 99) and beside(rooms, size // 32, 99)


@pytest.mark.parametrize("tokens", [1, 3, 5, 30, 1003])
@pytest.mark.parametrize("size", SIZES)
def test_act(tokens, size):
    x, up = inputs(tokens, size, F, 3, False), inputs(tokens, size, F, 4, False)
    x[0, 0] = 0.0
    for kind, second in (("silu", up), ("none", None), ("gelu", None)):
        y, e = ref.act(x, second, kind), ref.act_error(x, kind)
        room, out = guarded(tokens, size, torch.int8, 99)
        s = torch.empty(tokens, device="cuda")
        q.qgemm_act_quant(x, out, s, up=second, activation=kind)
        ref.check_int8(out, s, y, e)
        assert beside(room, size, 99)
        if size % 32 == 0:
            (room, out), (rooms, scales) = guarded(tokens, size, torch.uint8, 99), guarded(tokens, size // 32, torch.uint8, 99)
            q.qgemm_act_quant(x, out, scales, up=second, activation=kind)
            ref.check_e4m3(out, scales, y, e)
            assert beside(room, size, 99) and beside(rooms, size // 32, 99)


@pytest.mark.parametrize("size", [64, 128, 256])
def test_heads_in_place(size):
    """The heads of a projection's output, normed where they lie."""
    tokens, heads = 37, 3
    both = inputs(tokens, 2 * heads * size, B, 5, False)
    keep = both.clone()
    x = both[:, :heads * size].unflatten(1, (heads, size))
    for i in range(heads):
        q.qgemm_norm_quant(x[:, i], None, x[:, i], eps=1e-5)
        ref.check_16(x[:, i], ref.norm(keep[:, i * size:(i + 1) * size], None, None, 1e-5)[1], ref.norm_error(size))
    assert torch.equal(both[:, heads * size:], keep[:, heads * size:])


def test_nan_stays_in_its_row():
    for size in (64, 128, 256):
        x = inputs(16, size, B, 6, False)
        x[5, 3], x[9, 7] = float("nan"), float("inf")
        y, s = torch.empty(16, size, dtype=torch.int8, device="cuda"), torch.empty(16, device="cuda")
        q.qgemm_norm_quant(x, None, y, s, eps=1e-5)
        rest = [i for i in range(16) if i not in (5, 9)]
        ref.check_int8(y[rest], s[rest], ref.norm(x[rest], None, None, 1e-5)[1], ref.norm_error(size))
        assert not torch.isfinite(s[5]) and not torch.isfinite(s[9]) and not y[5].any() and not y[9].any()

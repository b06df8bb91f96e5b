"""Norm and activation with 8-bit output on the GPU against plain 64-bit forms."""
import math

import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

F, B = torch.float16, torch.bfloat16
# one element to past the vector kernel's longest row; multiples of 32, of 8 and neither; warps' and blocks' edges
SIZES = [1, 7, 8, 31, 32, 96, 250, 256, 1000, 1024, 1032, 2049, 4096, 5120, 8192, 14336, 16392, 28672, 32768, 32800, 40001]


def outputs(tokens, size, to, dtype, pad=0):
    """(Y, scales) of a format; rows `pad` elements longer than they need be."""
    if to == "16":
        return torch.full((tokens, size + pad), 7, dtype=dtype, device="cuda")[:, :size], None
    if to == "int8":
        return (torch.full((tokens, size + pad), 99, dtype=torch.int8, device="cuda")[:, :size],
                torch.full((tokens,), -5.0, device="cuda"))
    return (torch.full((tokens, size + pad), 99, dtype=torch.uint8, device="cuda")[:, :size],
            torch.full((tokens, size // 32 + pad), 99, dtype=torch.uint8, device="cuda")[:, :size // 32])


def check(y, s, want, to, e):
    if to == "int8":
        ref.check_int8(y, s, want, e)
    elif to == "e4m3":
        ref.check_e4m3(y, s, want, e)
    else:
        ref.check_16(y, want, e)


def rows(tokens, size, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, size, generator=g, device="cuda") * scale
    return (x * (1 + 15 * (torch.rand(size, generator=g, device="cuda") < 0.02))).to(dtype)


@pytest.mark.parametrize("to", ["int8", "e4m3", "16"])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("size", SIZES)
def test_norm(size, dtype, to):
    if to == "e4m3" and size % 32:
        pytest.skip("blocks of 32")
    tokens = 5
    x, r = rows(tokens, size, dtype, size), rows(tokens, size, dtype, size + 1, 2.0)
    w = rows(1, size, dtype, size + 2)[0]
    for residual, weight in ((r, w), (None, w.float()), (r, None)):
        y, s = outputs(tokens, size, to, dtype)
        h = torch.empty_like(x) if residual is not None else None
        q.qgemm_norm_quant(x, weight, y, s, residual=residual, residual_out=h, eps=1e-5)
        wh, wy = ref.norm(x, residual, weight, 1e-5)
        check(y, s, wy, to, ref.norm_error(size))
        if h is not None:
            ref.check_16(h, wh, ref.U32)


@pytest.mark.parametrize("kind,gated", [("none", False), ("none", True), ("silu", True), ("silu", False), ("gelu", True)])
@pytest.mark.parametrize("to", ["int8", "e4m3", "16"])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("size", SIZES[::2] + [14336])
def test_act(size, dtype, to, kind, gated):
    if to == "e4m3" and size % 32:
        pytest.skip("blocks of 32")
    tokens = 4
    both = rows(tokens, 2 * size, dtype, size, 2.0)
    x, up = both.split([size, size], 1)                  # the halves of a fused product's output
    up = up if gated else None
    y, s = outputs(tokens, size, to, dtype)
    q.qgemm_act_quant(x, y, s, up=up, activation=kind)
    check(y, s, ref.act(x, up, kind), to, ref.act_error(x, kind))


@pytest.mark.parametrize("tokens", [1, 2, 7, 153, 1000, 3001])
@pytest.mark.parametrize("size", [64, 520, 4096])
@pytest.mark.parametrize("to", ["int8", "e4m3", "16"])
def test_many_rows(tokens, size, to):
    """Rows beyond a block's first one, each with its own magnitude; nothing is written beside them."""
    if to == "e4m3" and size % 32:
        pytest.skip("blocks of 32")
    x = (rows(tokens, size, B, 3).float() * torch.exp2(torch.arange(tokens, device="cuda") % 40 - 20)[:, None]).to(B)
    y, s = outputs(tokens + 1, size, to, B, pad=8)
    y0, s0 = y[tokens].clone(), None if s is None else s[tokens].clone()
    edge = y._base[:, size:].clone()
    q.qgemm_norm_quant(x, None, y[:tokens], None if s is None else s[:tokens])
    check(y[:tokens], None if s is None else s[:tokens], ref.norm(x, None, None, 1e-6)[1], to, ref.norm_error(size))
    assert torch.equal(y[tokens], y0) and torch.equal(y._base[:, size:], edge)
    assert s is None or torch.equal(s[tokens], s0)


@pytest.mark.parametrize("off", [0, 1, 2, 4])
@pytest.mark.parametrize("to", ["int8", "e4m3", "16"])
def test_alignment(off, to):
    """Bases and strides of any alignment give the same bits as aligned ones of the same kernel's definition."""
    size, tokens = 544, 9
    x, r, w = rows(tokens, size, F, 1), rows(tokens, size, F, 2), rows(1, size, F, 3)[0]
    wide = size + off
    xs, rs = (torch.zeros(tokens * wide + off, dtype=F, device="cuda")[off:].view(tokens, wide)[:, :size] for _ in range(2))
    xs.copy_(x)
    rs.copy_(r)
    y, s = outputs(tokens, size, to, F, pad=off)
    q.qgemm_norm_quant(xs, w, y, s, residual=rs, residual_out=rs, eps=1e-6)
    h, want = ref.norm(x, r, w, 1e-6)
    check(y, s, want, to, ref.norm_error(size))
    ref.check_16(rs, h, ref.U32)


def test_repeated_rows_and_single_rows():
    x = rows(1, 512, B, 1).expand(6, 512)                # a row of stride 0
    y, s = outputs(6, 512, "int8", B)
    q.qgemm_act_quant(x, y, s)
    ref.check_int8(y, s, x.double(), 2 * ref.U32)
    assert torch.all(y == y[0]) and torch.all(s == s[0])
    odd = torch.as_strided(rows(1, 600, B, 2), (1, 512), (3, 1))    # a stride that is never stepped
    y, s = outputs(1, 512, "e4m3", B)
    q.qgemm_act_quant(odd, y, s)
    ref.check_e4m3(y, s, odd.double(), ref.U32)


@pytest.mark.parametrize("size", [512, 520, 515, 33000])
def test_in_place(size):
    x, r, w = rows(7, size, B, 1), rows(7, size, B, 2), rows(1, size, B, 3)[0]
    h, y = ref.norm(x, r, w, 1e-6)
    for target in ("x", "residual"):
        xs, rs = x.clone(), r.clone()
        out, s = outputs(7, size, "int8", B)
        q.qgemm_norm_quant(xs, w, out, s, residual=rs, residual_out=xs if target == "x" else rs, eps=1e-6)
        ref.check_int8(out, s, y, ref.norm_error(size))
        ref.check_16(xs if target == "x" else rs, h, ref.U32)
        assert torch.equal(rs if target == "x" else xs, r if target == "x" else x)
    xs, rs = x.clone(), r.clone()
    q.qgemm_norm_quant(xs, w, xs, residual=rs, residual_out=rs, eps=1e-6)
    ref.check_16(xs, y, ref.norm_error(size))
    both = torch.cat([x, r], 1)
    gate, up = both.split([size, size], 1)
    want = ref.act(gate, up, "silu")
    e = ref.act_error(gate, "silu")
    q.qgemm_act_quant(gate, gate, up=up, activation="silu")
    ref.check_16(gate, want, e)
    assert torch.equal(up, r)


@pytest.mark.parametrize("size", [96, 4096, 4101, 33024])
@pytest.mark.parametrize("dtype", [F, B])
def test_zero_rows(size, dtype):
    x = torch.zeros(3, size, dtype=dtype, device="cuda")
    x[1] = 1
    for run in (lambda y, s: q.qgemm_norm_quant(x, None, y, s, eps=1e-6), lambda y, s: q.qgemm_act_quant(x, y, s)):
        y, s = outputs(3, size, "int8", dtype)
        run(y, s)
        assert torch.all(y[0] == 0) and torch.all(y[2] == 0) and torch.all(y[1] == 127)
        assert float(s[0]) == float(torch.tensor(ref.LEAST / 127, dtype=torch.float32))
        if size % 32 == 0:
            y, s = outputs(3, size, "e4m3", dtype)
            run(y, s)
            assert torch.all(y[0] == 0) and torch.all(s[0] == 127)


@pytest.mark.parametrize("size", [256, 4096, 4100, 33024])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e15, 1e18, 1e25, 3e37])
def test_range(size, scale):
    """bfloat16 rows up to the type's end: sums of squares past fp32's range; and down to where eps decides."""
    x = rows(4, size, B, 5, 0.05).clamp(-1, 1).float().mul(scale).to(B)
    x[0] = 0
    x[0, 3] = scale
    w = rows(1, size, B, 6)[0]
    want = ref.norm(x, None, w, 1e-6)[1]
    # past the range eps is left out: below 2^-140 of the mean
    for to in ("int8", "16", "e4m3"):
        if to == "e4m3" and size % 32:
            continue
        y, s = outputs(4, size, to, B)
        q.qgemm_norm_quant(x, w, y, s, eps=1e-6)
        check(y, s, want, to, ref.norm_error(size) + 2.0 ** -20)   # r may be an fp32 subnormal of 21 bits


@pytest.mark.parametrize("size", [256, 4096, 4097, 33024])
def test_nan_and_infinity(size):
    x = rows(5, size, B, 7)
    x[1, size // 2] = math.nan
    x[2, size - 1] = math.inf
    x[3, 0] = -math.inf
    x[3, 1] = math.nan
    y, s = outputs(5, size, "int8", B)
    q.qgemm_act_quant(x, y, s)
    ref.check_int8(y[[0, 4]], s[[0, 4]], x[[0, 4]].double(), 2 * ref.U32)
    assert s[1].isnan() and s[2] == math.inf and s[3].isnan()
    assert torch.all(y[1:4] == 0)
    q.qgemm_norm_quant(x, None, y, s, eps=1e-6)
    ref.check_int8(y[[0, 4]], s[[0, 4]], ref.norm(x[[0, 4]], None, None, 1e-6)[1], ref.norm_error(size))
    assert torch.all(s[1:4].isnan())                     # an infinite h over an infinite norm
    out, _ = outputs(5, size, "16", B)
    q.qgemm_norm_quant(x, None, out, eps=1e-6)
    assert torch.all(out[1].isnan()) and out[2, -1].isnan() and torch.all(out[2, :-1] == 0) and torch.all(out[3].isnan())
    if size % 32 == 0:
        y, s = outputs(5, size, "e4m3", B)
        q.qgemm_act_quant(x, y, s)
        v = y.view(torch.float8_e4m3fn).float()
        assert v[1, size // 2].isnan() and int(v[1].isnan().sum()) == 1
        assert v[2, -1] == 448 and s[2, -1] == 247 and v[3, 0] == -448 and v[3, 1].isnan() and s[3, 0] == 247
        ref.check_e4m3(y[[0, 4]], s[[0, 4]], x[[0, 4]].double(), ref.U32)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [F, B])
def test_act_far_from_zero(kind, dtype):
    """exp overflows for large negative arguments: the result goes to zero as the type's range does, without a NaN."""
    v = torch.tensor([-60000.0, -1000.0, -120.0, -89.0, -88.0, -20.0, -1.0, 0.0, 1.0, 20.0, 1000.0, 60000.0], dtype=dtype, device="cuda")
    x = v.repeat(2, 8)
    y, _ = outputs(2, 96, "16", dtype)
    q.qgemm_act_quant(x, y, activation=kind)
    ref.check_16(y, ref.act(x, None, kind), ref.act_error(x, kind))
    big = torch.full((1, 96), 3e38, dtype=B, device="cuda")
    y, _ = outputs(1, 96, "16", B)
    q.qgemm_act_quant(big, y, activation=kind)
    assert torch.equal(y, big)
    q.qgemm_act_quant(-big, y, activation=kind)
    assert torch.all(y == 0)


def test_repeatable():
    x, r, w = rows(3001, 4096, B, 1), rows(3001, 4096, B, 2), rows(1, 4096, B, 3)[0]
    first = None
    for _ in range(3):
        y, s = outputs(3001, 4096, "int8", B)
        h = torch.empty_like(x)
        q.qgemm_norm_quant(x, w, y, s, residual=r, residual_out=h)
        if first is not None:
            assert torch.equal(y, first[0]) and torch.equal(s, first[1]) and torch.equal(h, first[2])
        first = (y, s, h)


def test_no_rows():
    x = torch.empty(0, 64, dtype=F, device="cuda")
    y, s = outputs(0, 64, "int8", F)
    q.qgemm_act_quant(x, y, s)
    q.qgemm_norm_quant(x, None, y, s)


@pytest.mark.parametrize("size", [512, 4096, 4101, 33000])
def test_ties(size):
    """Values exactly half-way between two codes go to the even one: halves of a row's largest, whatever that is."""
    tokens = 200
    top = (1 + torch.arange(tokens, device="cuda") / 128).clamp(max=1.9921875).to(B)       # every bf16 significand
    x = torch.zeros(tokens, size, dtype=B, device="cuda")
    x[:, 0] = top
    odd = torch.arange(1, 127, 2, device="cuda", dtype=torch.float64) / 2                    # 0.5, 1.5, ... codes
    for k, code in enumerate(odd.tolist()):
        v = top.double() * code / 127
        x[:, 1 + k] = torch.where(v.to(B).double() == v, v, 0).to(B)
    x[:, -1] = -(top.double() / 2).to(B)                                                     # -63.5
    y, s = outputs(tokens, size, "int8", B)
    q.qgemm_act_quant(x, y, s)
    want = torch.round(x.double() * 127 / top.double()[:, None])
    assert torch.equal(y.double(), want)
    assert torch.all(y[:, -1] == -64)

"""Host-side checks of the 8-bit linear layers' calls (no GPU): refusals before anything is enqueued."""
import ctypes

import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from block_scaled_quantized_tcgen05_gb300 import build as qbuild

P = ctypes.c_void_p
OK, INVALID, SHAPE, MISALIGNED, DTYPE, CUDA = 0, 1, 2, 3, 4, 5
X, R, RO, W, Y, S = (0x100000 * (i + 1) for i in range(6))
NORM = dict(x=X, ldx=64, r=R, ldr=64, ro=RO, ldro=64, dt=q.F16, w=W, wdt=q.F32, eps=1e-6, T=4, H=64, y=Y, ldy=64, ydt=q.INT8, s=S,
            lds=2)
ACT = dict(x=X, ldx=128, u=X + 128, ldu=128, dt=q.BF16, kind=1, T=4, H=64, y=Y, ldy=64, ydt=q.E4M3, s=S, lds=2)
PROD = dict(a=X, lda=64, sa=S, w=W, ldw=64, sw=S, bias=R, c=Y, ldc=48, dt=q.F16, M=4, N=48, K=50)


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.load_library()


def call(lib, base, **change):
    a = dict(base, **change)
    fn = {id(NORM): lib.qgemm_norm_quant, id(ACT): lib.qgemm_act_quant, id(PROD): lib.qgemm_w8a8}[id(base)]
    pointers = {"x", "r", "ro", "w", "y", "s", "u", "a", "sa", "sw", "bias", "c"}
    return fn(*(P(v or None) if k in pointers else v for k, v in a.items()), None)


def refused(lib, base, status, **change):
    assert call(lib, base, **change) == status, (change, lib.qgemm_last_error_message())


BIG = 1 << 31


@pytest.mark.parametrize("change,status", [
    ({"x": 0}, INVALID), ({"y": 0}, INVALID), ({"s": 0}, INVALID), ({"r": 0}, INVALID), ({"T": -1}, INVALID), ({"H": -1}, INVALID),
    ({"eps": 0.0}, INVALID), ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID), ({"eps": float("inf")}, INVALID),
    ({"eps": 1e39}, INVALID), ({"eps": 2.0 ** -65}, INVALID), ({"dt": q.F32}, DTYPE), ({"dt": q.INT8}, DTYPE), ({"wdt": q.INT8}, DTYPE),
    ({"ydt": q.BF16}, DTYPE), ({"ydt": q.F32}, DTYPE), ({"ydt": q.INT4}, DTYPE), ({"T": BIG}, SHAPE), ({"H": BIG}, SHAPE),
    ({"ydt": q.E4M3, "H": 63}, SHAPE), ({"ldx": -64}, INVALID), ({"ldr": -1}, INVALID), ({"ldro": 63}, INVALID), ({"ldy": 63}, INVALID),
    ({"ydt": q.E4M3, "lds": 1}, INVALID), ({"x": X + 1}, MISALIGNED), ({"r": R + 1}, MISALIGNED), ({"ro": RO + 1}, MISALIGNED),
    ({"w": W + 2}, MISALIGNED), ({"s": S + 2}, MISALIGNED), ({"ydt": q.F16}, INVALID), ({"ydt": q.F16, "s": 0, "y": Y + 1}, MISALIGNED),
    ({"ldx": 1 << 60}, INVALID), ({"ldy": 1 << 60}, INVALID),
    # outputs that lie over other operands
    ({"ro": X + 2}, INVALID), ({"ro": R, "ldr": 65}, INVALID), ({"ro": Y}, INVALID), ({"y": X}, INVALID), ({"y": R + 64}, INVALID),
    ({"ydt": q.F16, "s": 0, "y": RO}, INVALID), ({"ydt": q.F16, "s": 0, "y": X + 128 * 3}, INVALID),
])
def test_norm_refusals(lib, change, status):
    refused(lib, NORM, status, **change)


@pytest.mark.parametrize("change,status", [
    ({"x": 0}, INVALID), ({"y": 0}, INVALID), ({"s": 0}, INVALID), ({"kind": 3}, INVALID), ({"kind": -1}, INVALID), ({"dt": q.E4M3}, DTYPE),
    ({"ydt": q.F16}, DTYPE), ({"H": 65, "ldy": 65}, SHAPE), ({"u": X + 129}, MISALIGNED), ({"x": X + 1}, MISALIGNED), ({"ldu": -2}, INVALID),
    ({"lds": 1}, INVALID), ({"y": X + 64}, INVALID), ({"ydt": q.BF16, "s": 0, "y": X + 64, "ldy": 128}, INVALID),
    ({"ydt": q.BF16, "s": 0, "y": X, "ldy": 64}, INVALID), ({"T": BIG}, SHAPE),
])
def test_act_refusals(lib, change, status):
    refused(lib, ACT, status, **change)


@pytest.mark.parametrize("change,status", [
    ({"a": 0}, INVALID), ({"w": 0}, INVALID), ({"sa": 0}, INVALID), ({"sw": 0}, INVALID), ({"c": 0}, INVALID), ({"M": -1}, INVALID),
    ({"N": -1}, INVALID), ({"K": -1}, INVALID), ({"M": BIG}, SHAPE), ({"N": BIG}, SHAPE), ({"K": BIG}, SHAPE), ({"dt": q.F32}, DTYPE),
    ({"dt": q.INT8}, DTYPE), ({"lda": 48}, INVALID), ({"ldw": 48}, INVALID), ({"lda": 56}, MISALIGNED), ({"ldw": 72}, MISALIGNED),
    ({"a": X + 8}, MISALIGNED), ({"w": W + 8}, MISALIGNED), ({"sa": S + 2}, MISALIGNED), ({"sw": S + 1}, MISALIGNED), ({"c": Y + 1}, MISALIGNED),
    ({"bias": R + 1}, MISALIGNED), ({"ldc": 47}, INVALID), ({"lda": 1 << 60}, INVALID), ({"ldw": 1 << 40}, SHAPE),
])
def test_product_refusals(lib, change, status):
    refused(lib, PROD, status, **change)


@pytest.mark.parametrize("change", [{"M": BIG - 4095}, {"N": BIG - 4095, "ldc": BIG}, {"K": BIG - 4095, "lda": BIG, "ldw": BIG}])
def test_product_sizes_round_up_in_31_bits(lib, change):
    """The kernels round sizes up to whole tiles in 32-bit integers."""
    refused(lib, PROD, SHAPE, **change)


def test_epilogue_fields(lib):
    for bad in ((2, 0), (0, -1)):
        ep = q.Epilogue(*bad)
        assert lib.qgemm_w8a8_ex(P(X), 64, P(S), P(W), 64, P(S), None, P(Y), 48, 0, 4, 48, 50, ctypes.byref(ep), None) == INVALID


@pytest.mark.parametrize("base,change", [
    (NORM, {}), (NORM, {"ro": X}), (NORM, {"ro": R}), (NORM, {"r": 0, "ro": 0}), (NORM, {"w": 0}), (NORM, {"T": 1, "ldx": -7, "ldy": 0}),
    (NORM, {"ydt": q.F16, "s": 0, "y": X}), (NORM, {"ydt": q.F16, "s": 0, "y": R}), (NORM, {"ldx": 0}), (NORM, {"eps": 2.0 ** -64}),
    # halves of fused buffers lie between each other's rows
    (NORM, {"x": X, "ldx": 128, "ro": X + 128, "ldro": 128}), (NORM, {"x": X + 128, "ldx": 128, "ro": X, "ldro": 128}),
    (ACT, {}), (ACT, {"u": 0}), (ACT, {"ydt": q.BF16, "s": 0, "y": X, "ldy": 128}), (ACT, {"ydt": q.BF16, "s": 0, "y": X + 128, "ldy": 128}),
    (PROD, {}), (PROD, {"bias": 0}), (PROD, {"K": 64}), (PROD, {"M": 1, "lda": 0, "ldc": 0}), (PROD, {"K": 0, "a": 0, "w": 0, "sa": 0, "sw": 0}),
])
def test_allowed(lib, base, change):
    """What is allowed gets as far as the device, which is not there."""
    if torch.cuda.is_available():
        pytest.skip("would launch")
    refused(lib, base, CUDA, **change)


@pytest.mark.parametrize("base,change", [(NORM, {"T": 0}), (NORM, {"H": 0}), (ACT, {"T": 0, "x": 0}), (PROD, {"M": 0}), (PROD, {"N": 0, "c": 0})])
def test_nothing_to_do(lib, base, change):
    refused(lib, base, OK, **change)


def test_binding_refuses_what_it_can_see():
    x = torch.zeros(4, 64, dtype=torch.float16)
    y, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="current device"):
        q.qgemm_act_quant(x, y, s)
    with pytest.raises(ValueError, match="current device"):
        q.qgemm_norm_quant(x, None, y, s)
    with pytest.raises(ValueError, match="activation"):
        q.qgemm_act_quant(x, y, s, activation="relu")
    with pytest.raises(ValueError, match="int8"):
        q.qgemm_w8a8(x, s, y, s, x)
    with pytest.raises(ValueError, match="contiguous rows"):
        q.qgemm_act_quant(x.t(), y.t(), s)

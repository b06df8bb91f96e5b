"""Plain 64-bit forms of the 8-bit linear layers' operators, and the bounds their kernels are held to.

The bounds count roundings: U32 = 2^-24 for fp32, torch.finfo(t).eps / 2 for a 16-bit output, half a step for a code.
"""
import math

import torch

U32 = 2.0 ** -24
LEAST = 2.0 ** -100


def norm(x, residual, weight, eps):
    """(h, y) in 64 bits."""
    h = x.double() if residual is None else x.double() + residual.double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return h, y if weight is None else y * weight.double()


def act(x, up, kind):
    y = x.double()
    if kind == "silu":
        y = y * torch.sigmoid(y)
    elif kind == "gelu":
        # (1 + tanh u) / 2 as sigmoid(2 u): 1 + tanh u cancels for negative u, in 64 bits from u = -18 on altogether
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    return y if up is None else y * up.double()


def norm_error(size):
    """Relative error of y in fp32: h, a sum of `size` squares (at worst one after another in a thread's share of a
    256th, then 10 joins), the mean, rsqrt (2 units), three products."""
    return (size / 256 + 10 + 12) * U32


def act_error(x, kind="gelu"):
    """Relative error of f(x) * up in fp32: exp(-v) through the base-2 exponential carries v's relative error |v| times.
    v is x itself for silu and 2 roundings old with the factor log2(e); for gelu v = 2 u, |v| <= 1.6 |x| (1 + x^2 / 22), with 7
    more roundings.  Past 104 exp(-|v|) is 0 in fp32 for every such error.  The exponential (2 units, twice as a
    square: 8), the reciprocal (1 unit: 2), the sum and five products add at most 16."""
    top = float(x.abs().max())
    v = top if kind != "gelu" else 1.6 * top * (1 + top * top / 22)
    return ((9 if kind == "gelu" else 2) * min(104.0, v) + 16) * U32


def check_int8(q, s, y, e):
    """Codes and scales against y (64 bits) known to the kernel within a relative error of e."""
    amax = y.abs().amax(-1).clamp(min=LEAST)
    want = amax / 127
    assert torch.all((s.double() - want).abs() <= want * (e + 2 * U32) * 1.01 + 2.0 ** -149), "scale"
    off = (q.double() - y / want[:, None]).abs()
    # half a step, and what y's and the factor's errors (e each, and two roundings) move a value of at most 127
    assert float(off.max()) <= 0.5 + 127 * (2 * e + 3 * U32), float(off.max())


def check_e4m3(codes, bytes_, y, e):
    """E4M3 codes and UE8M0 bytes against y (64 bits) known within a relative error of e."""
    b = y.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    x = bytes_.double() - 127
    low = torch.floor(torch.log2(torch.where(amax > 0, amax * (1 - e), 256.0))) - 8
    high = torch.floor(torch.log2(torch.where(amax > 0, amax * (1 + e), 256.0))) - 8
    low, high = low.clamp(min=-127.0), high.clamp(min=-127.0)
    assert torch.all((x == low) | (x == high)), "scale byte"
    v = codes.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
    r = (b * torch.exp2(-x)[..., None]).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2((r.abs() * (1 + e)).clamp(min=2.0 ** -6))) - 3)
    bad = (v - r).abs() > step / 2 + e * r.abs()
    assert not bad.any(), (v[bad][:4], r[bad][:4])


def check_16(out, y, e):
    """A 16-bit output: half a unit of its type (its subnormals' half step at least) beside the error e."""
    info = torch.finfo(out.dtype)
    bound = y.abs() * (info.eps / 2 + 2 * e) + info.smallest_normal * info.eps
    assert torch.all((out.double() - y).abs() <= bound), float(((out.double() - y).abs() / bound).max())


def product(a, sa, w, sw, bias=None, old=None, relu=False):
    """(C, sum of the products' magnitudes times the scales) in 64 bits; integer sums are exact (below 2^53)."""
    scale = sa.double()[:, None] * sw.double()
    y = (a.double() @ w.double().T) * scale
    size = (a.double().abs() @ w.double().abs().T) * scale.abs()
    for more in (bias, old):
        if more is not None:
            y = y + more.double()
            size = size + more.double().abs()
    return y.clamp(min=0) if relu else y, size


def product_error(k, top):
    """Bound on the error relative to the sum of magnitudes: integer sums are exact while they stay below 2^24
    (`top`, their largest possible magnitude); past it each of the k / 16 accumulations may lose a unit, at most 2^-23 as
    the tensor cores cut.  Two scale products, a bias and an old output round once each."""
    return (0.0 if top < 2 ** 24 else (k / 16 + 1) * 2 * U32) + 5 * U32


def check_product(out, y, size, k, top):
    info = torch.finfo(out.dtype)
    bound = y.abs() * info.eps / 2 * 1.01 + size * product_error(k, top) * 1.01 + info.smallest_normal * info.eps
    far = (out.double() - y).abs()
    assert torch.all(far <= bound), float((far / bound).max())

"""Workloads of the 8-bit linear layers' operators: the root-mean-square norm (with the residual's
addition) and the gated activation that leave 8 bits with scales, and the matrix product of 8-bit
integers with a scale for each token and each channel.

`run` computes a workload either with the library (`own` true) or in plain torch operations in 32
bits; `exact` restates it in 64 bits.  Sizes are those of the library's own products (4096, 8192,
14336, 28672) and generic ones around them.

Eight bits are one of two formats: "int8", with one fp32 scale for each token, or "e4m3", with one
UE8M0 scale for each 32 elements, as the library's block-scaled products take them.  Integer codes
are returned as 16-bit floats, E4M3 codes and UE8M0 scales as the numbers they stand for.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32
EPS = 1e-6
LEAST = 2.0 ** -100  # the least magnitude an integer row's scale is taken from
DEV = "cuda"


def listed():
    return [
        # one decode step's norm before a projection, 8 sequences: latency
        norm_case(8, 4096, "f16", "e4m3", True, name="norm_decode_8"),
        # a prefill chunk before a block-scaled product
        norm_case(8192, 8192, "bf16", "e4m3", True, name="norm_prefill_8192"),
        # odd token count and a row that is no multiple of the vector width, first layer (no residual)
        norm_case(5003, 5111, "bf16", "int8", False, name="norm_int8_odd"),
        # one decode step's gated activation, 16 sequences: latency
        act_case(16, 14336, "bf16", "silu", True, "int8", name="act_decode_16"),
        # a prefill chunk's gated activation before the product back
        act_case(4096, 14336, "f16", "silu", True, "e4m3", name="act_prefill_4096"),
        # the attention's output (no activation), an odd token count
        act_case(6007, 4096, "bf16", "none", False, "int8", name="act_attention_odd"),
        # one sequence's decode step: latency, the weights' bytes
        product_case(1, 28672, 8192, "f16", False, name="product_1x28672x8192"),
        # a small serving batch, a square projection
        product_case(8, 4096, 4096, "bf16", True, name="product_8x4096x4096"),
        # a larger serving batch: the weights' bytes still
        product_case(64, 28672, 8192, "bf16", False, name="product_64x28672x8192"),
        # ragged: no size a multiple of a tile, rows of weights padded to 16 bytes
        product_case(333, 5003, 4111, "f16", True, name="product_ragged_333"),
        # a prefill chunk
        product_case(4096, 14336, 4096, "f16", False, name="product_4096x14336x4096"),
        # the largest
        product_case(8192, 8192, 8192, "bf16", False, name="product_8192"),
    ]


def norm_case(tokens, size, dtype, to, residual, **more):
    return dict(more, op="norm", tokens=tokens, size=size, dtype=dtype, to=to, residual=residual)


def act_case(tokens, size, dtype, kind, gated, to, **more):
    """`gated`: the activation of the first half of a row times the second half, as a fused product leaves them."""
    return dict(more, op="act", tokens=tokens, size=size, dtype=dtype, kind=kind, gated=gated, to=to)


def product_case(m, n, k, dtype, bias, **more):
    return dict(more, op="product", m=m, n=n, k=k, dtype=dtype, bias=bias)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "act", "product", "product"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "product":
        m, n = log(1, 8192), log(16, 28672)
        k = log(16, min(28672, 8192 ** 3 // (m * n)))
        if rng.random() < 0.6:
            n, k = -(-n // 128) * 128, -(-k // 128) * 128
        return product_case(m, n, k, dtype, rng.random() < 0.5)
    to = rng.choice(["int8", "e4m3"])
    size = log(32, 28672)
    if to == "e4m3" or rng.random() < 0.6:
        size = -(-size // BLOCK) * BLOCK
    tokens = log(1, min(16384, 2 ** 26 // size))
    if op == "norm":
        return norm_case(tokens, size, dtype, to, rng.random() < 0.7)
    kind = rng.choice(["none", "silu", "silu", "gelu"])
    return act_case(tokens, size, dtype, kind, kind != "none", to)


def work(c):
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": m * k + n * k + 4 * m + 4 * n + 2 * m * n + (2 * n if c["bias"] else 0), "flops": 2 * m * n * k}
    t, h = c["tokens"], c["size"]
    out = t * (h + 4) if c["to"] == "int8" else t * (h + h // BLOCK)
    if c["op"] == "norm":
        return {"bytes": t * h * (6 if c["residual"] else 2) + 2 * h + out, "flops": 6 * t * h}
    return {"bytes": t * h * (4 if c["gated"] else 2) + out, "flops": (12 if c["gated"] else 2) * t * h}


# ------------------------------------------------------------------------------------ inputs

def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"norm": prepare_norm, "act": prepare_act, "product": prepare_product}[c["op"]](dict(c), g)


def normal(shape, dtype, g, strong=0.01):
    """Activations: of unit size, a few channels much stronger than the rest."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    x *= (1 + 15 * (torch.rand(shape[-1], generator=g, device=DEV) < strong)).to(dtype)
    return x


def outputs(c):
    """The output's codes and scales, as a program keeps them between calls."""
    t, h = c["tokens"], c["size"]
    if c["to"] == "int8":
        room = torch.empty(t, -(-h // 16) * 16, dtype=torch.int8, device=DEV)  # rows as the product takes them
        return {"y": room[:, :h], "s": torch.empty(t, dtype=torch.float32, device=DEV)}
    return {"y": torch.empty(t, h, dtype=torch.uint8, device=DEV), "s": torch.empty(t, h // BLOCK, dtype=torch.uint8, device=DEV)}


def prepare_norm(c, g):
    shape, dt = (c["tokens"], c["size"]), TYPES[c["dtype"]]
    s = {"c": c, "x": normal(shape, dt, g), **outputs(c)}
    s["w"] = (1 + 0.2 * torch.randn(c["size"], generator=g, device=DEV)).to(dt)
    if c["residual"]:
        s["r"] = 3 * normal(shape, dt, g)
        s["h"] = torch.empty_like(s["r"])
    return s


def prepare_act(c, g):
    t, h, dt = c["tokens"], c["size"], TYPES[c["dtype"]]
    s = {"c": c, **outputs(c)}
    if c["gated"]:
        s["x"], s["up"] = normal((t, 2 * h), dt, g).mul_(2).split([h, h], 1)
    else:
        s["x"], s["up"] = normal((t, h), dt, g), None
    return s


def codes_of(x, room):
    """The integer codes and the scales of x's rows (through `room`, whose rows are padded to 16 bytes)."""
    scale = x.abs().amax(1).float().clamp(min=LEAST) / 127
    room[:, :x.shape[1]] = torch.round(x / scale[:, None].to(x.dtype)).clamp(-127, 127).to(torch.int8)
    return room[:, :x.shape[1]], scale


def prepare_product(c, g):
    m, n, k, dt = c["m"], c["n"], c["k"], TYPES[c["dtype"]]
    width = -(-k // 16) * 16
    s = {"c": c}
    s["a"], s["sa"] = codes_of(normal((m, k), torch.float32, g), torch.zeros(m, width, dtype=torch.int8, device=DEV))
    s["w"], s["sw"] = codes_of(0.02 * torch.randn(n, k, generator=g, device=DEV), torch.zeros(n, width, dtype=torch.int8, device=DEV))
    s["bias"] = torch.randn(n, generator=g, device=DEV).to(dt) if c["bias"] else None
    s["y"] = torch.empty(m, n, dtype=dt, device=DEV)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    op = s["c"]["op"]
    if own:
        return {"norm": own_norm, "act": own_act, "product": own_product}[op](s)
    return {"norm": plain_norm, "act": plain_act, "product": plain_product}[op](s)


def numbers(s):
    """Codes and scales as the numbers they stand for."""
    if s["c"]["to"] == "int8":
        return {"y": s["y"].to(torch.float16), "s": s["s"]}
    return {"y": s["y"].view(torch.float8_e4m3fn), "s": s["s"].view(torch.float8_e8m0fnu)}


def own_norm(s):
    import block_scaled_quantized_tcgen05_gb300 as q
    q.qgemm_norm_quant(s["x"], s["w"], s["y"], s["s"], residual=s.get("r"), residual_out=s.get("h"), eps=EPS)
    return dict(numbers(s), h=s["h"]) if "r" in s else numbers(s)


def own_act(s):
    import block_scaled_quantized_tcgen05_gb300 as q
    q.qgemm_act_quant(s["x"], s["y"], s["s"], up=s["up"], activation=s["c"]["kind"])
    return numbers(s)


def own_product(s):
    import block_scaled_quantized_tcgen05_gb300 as q
    return q.qgemm_w8a8(s["a"], s["sa"], s["w"], s["sw"], s["y"], bias=s["bias"])


def to_eight_bits(s, y):
    """y (32 bits) as codes and scales, in the state's buffers."""
    if s["c"]["to"] == "int8":
        most = y.abs().amax(1).clamp(min=LEAST)
        codes = torch.round(y * (127 / most)[:, None]).clamp(-127, 127)
        s["y"].copy_(codes)
        s["s"].copy_(most / 127)
    else:
        b = y.unflatten(1, (-1, BLOCK))
        most = b.abs().amax(2)
        e = torch.where(most > 0, torch.frexp(most)[1] - 9, 0).clamp(-127, 127)
        s["y"].copy_(torch.ldexp(b, -e[..., None]).clamp(-448, 448).flatten(1).to(torch.float8_e4m3fn).view(torch.uint8))
        s["s"].copy_((e + 127).to(torch.uint8))
    return numbers(s)


def plain_norm(s):
    x = s["x"].float()
    if "r" in s:
        x = x + s["r"].float()
        s["h"].copy_(x)
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    return dict(to_eight_bits(s, y), h=s["h"]) if "r" in s else to_eight_bits(s, y)


def plain_act(s):
    y, kind = s["x"].float(), s["c"]["kind"]
    if kind == "silu":
        y = y / (1 + torch.exp(-y))
    elif kind == "gelu":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["up"] is not None:
        y = y * s["up"].float()
    return to_eight_bits(s, y)


def plain_product(s):
    y = (s["a"].float() @ s["w"].float().T) * s["sa"][:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    s["y"].copy_(y)
    return s["y"]


# ------------------------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "product":
        rows = [s["a"][i:i + 1024].double() @ s["w"].double().T for i in range(0, c["m"], 1024)]
        y = torch.cat(rows) * torch.outer(s["sa"].double(), s["sw"].double())
        return y if s["bias"] is None else y + s["bias"].double()
    got = {}
    x = s["x"].double()
    if c["op"] == "norm":
        if c["residual"]:
            x = x + s["r"].double()
            got["h"] = x
        length = torch.linalg.vector_norm(x, dim=1, keepdim=True)
        x = x / torch.sqrt(length * length / c["size"] + EPS) * s["w"].double()
    else:
        if c["kind"] == "silu":
            x = x * torch.sigmoid(x)
        elif c["kind"] == "gelu":
            x = x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
        if c["gated"]:
            x = x * s["up"].double()
    if c["to"] == "int8":
        scale = torch.clamp(x.abs().max(1)[0], min=LEAST) / 127
        return dict(got, y=torch.round(x / scale[:, None]), s=scale)
    blocks = x.reshape(c["tokens"], -1, BLOCK)
    top = blocks.abs().max(2)[0]
    unit = torch.exp2((torch.floor(torch.log2(torch.where(top > 0, top, 256.0))) - 8).clamp(min=-127.0))
    r = (blocks / unit[..., None]).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)
    return dict(got, y=(torch.round(r / step) * step).reshape(c["tokens"], c["size"]), s=unit)

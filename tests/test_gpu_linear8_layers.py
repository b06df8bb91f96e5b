"""The 8-bit linear layers' operators together: a transformer block's calls one after another, each checked on what the
one before it left, the chain to the block-scaled product, graphs, streams, and the example."""
import importlib.util
import os

import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import linear8_reference as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F, B = torch.float16, torch.bfloat16


def randn(*shape, seed=0, dtype=F, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def channels(w):
    codes, scales = torch.empty(w.shape, dtype=torch.int8, device="cuda"), torch.empty(w.shape[0], device="cuda")
    q.qgemm_act_quant(w, codes, scales)
    ref.check_int8(codes, scales, w.double(), 2 * ref.U32)
    return codes, scales


def product(a, s, w, bias=None, dtype=F):
    c = torch.empty(a.shape[0], w[0].shape[0], dtype=dtype, device="cuda")
    q.qgemm_w8a8(a, s, *w, c, bias=bias)
    y, size = ref.product(a, s, *w, bias)
    ref.check_product(c, y, size, a.shape[1], a.shape[1] * 127 ** 2)
    return c


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("tokens", [1, 7, 40, 300])
def test_block(tokens, dtype):
    hidden, mlp = 768, 2048
    wqkv, wo = channels(randn(1152, hidden, seed=1, scale=0.03, dtype=dtype)), channels(randn(hidden, hidden, seed=2, scale=0.03, dtype=dtype))
    wgu, wd = channels(randn(2 * mlp, hidden, seed=3, scale=0.03, dtype=dtype)), channels(randn(hidden, mlp, seed=4, scale=0.03, dtype=dtype))
    gain, bias = 1 + randn(hidden, seed=5, scale=0.1, dtype=torch.float32), randn(1152, seed=6, dtype=dtype)
    x, h = randn(tokens, hidden, seed=7, dtype=dtype), randn(tokens, hidden, seed=8, dtype=dtype)
    a, s = torch.empty(tokens, hidden, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
    wh, wy = ref.norm(x, h, gain, 1e-6)
    q.qgemm_norm_quant(x, gain, a, s, residual=h, residual_out=h)
    ref.check_16(h, wh, ref.U32)
    ref.check_int8(a, s, wy, ref.norm_error(hidden))
    qkv = product(a, s, wqkv, bias, dtype)
    mixed = qkv[:, :hidden]                               # in the attention's place: a slice of a wider buffer
    q.qgemm_act_quant(mixed, a, s)
    ref.check_int8(a, s, mixed.double(), 2 * ref.U32)
    y = product(a, s, wo, None, dtype)
    before = h.clone()
    q.qgemm_norm_quant(y, gain, a, s, residual=h, residual_out=h)
    wh, wy = ref.norm(y, before, gain, 1e-6)
    ref.check_16(h, wh, ref.U32)
    ref.check_int8(a, s, wy, ref.norm_error(hidden))
    gate, up = product(a, s, wgu, None, dtype).split([mlp, mlp], 1)
    a2 = torch.empty(tokens, mlp, dtype=torch.int8, device="cuda")
    q.qgemm_act_quant(gate, a2, s, up=up, activation="silu")
    ref.check_int8(a2, s, ref.act(gate, up, "silu"), ref.act_error(gate, "silu"))
    old = h.clone()
    q.qgemm_w8a8_ex(a2, s, *wd, h, accumulate=True)       # the residual's addition in the product's epilogue
    yy, size = ref.product(a2, s, *wd, None, old)
    ref.check_product(h, yy, size, mlp, mlp * 127 ** 2)
    assert q.qgemm_poll_device_error() == 0


@pytest.mark.parametrize("tokens", [5, 130])
def test_block_scaled_chain(tokens):
    """The E4M3 output is what the block-scaled product takes."""
    hidden, n = 512, 384
    x, r, gain = randn(tokens, hidden, seed=1), randn(tokens, hidden, seed=2), randn(hidden, seed=3)
    codes = torch.empty(tokens, hidden, dtype=torch.uint8, device="cuda")
    scales = torch.empty(tokens, hidden // 32, dtype=torch.uint8, device="cuda")
    q.qgemm_norm_quant(x, gain, codes, scales, residual=r, residual_out=r)
    w = randn(n, hidden, seed=4, scale=0.05)
    wcodes, wscales = torch.empty(n, hidden, dtype=torch.uint8, device="cuda"), torch.empty(n, hidden // 32, dtype=torch.uint8, device="cuda")
    q.qgemm_act_quant(w, wcodes, wscales)
    ref.check_e4m3(wcodes, wscales, w.double(), ref.U32)

    def values(c, s):
        return c.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).repeat_interleave(32, 1)

    c = torch.empty(tokens, n, dtype=F, device="cuda")
    q.qgemm_mxfp8(q.qgemm_create_tensor(q.E4M3, codes, scales), q.qgemm_create_tensor(q.E4M3, wcodes, wscales), c)
    a, b = values(codes, scales), values(wcodes, wscales)
    want, size = a @ b.T, a.abs() @ b.abs().T
    # fp32 sums of 512 products (a unit of 2^-23 lost for each 32 at worst), one fp16 rounding
    assert torch.all((c.double() - want).abs() <= want.abs() * 2.0 ** -11 + size * 17 * 2.0 ** -23 + 2.0 ** -25)


class Chain:
    """Buffers of norm -> product -> activation -> product, as a program captures them."""

    def __init__(self, tokens, seed):
        self.x, self.h = randn(tokens, 1024, seed=seed), randn(tokens, 1024, seed=seed + 1)
        self.w1, self.w2 = channels(randn(2 * 1536, 1024, seed=3, scale=0.03)), channels(randn(1000, 1536, seed=4, scale=0.03))
        self.a, self.s = torch.empty(tokens, 1024, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
        self.y1 = torch.empty(tokens, 2 * 1536, dtype=F, device="cuda")
        self.a2, self.s2 = torch.empty(tokens, 1536, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
        self.y2 = torch.empty(tokens, 1000, dtype=F, device="cuda")

    def run(self, stream=None):
        q.qgemm_norm_quant(self.x, None, self.a, self.s, residual=self.h, stream=stream)
        q.qgemm_w8a8(self.a, self.s, *self.w1, self.y1, stream=stream)
        q.qgemm_act_quant(self.y1[:, :1536], self.a2, self.s2, up=self.y1[:, 1536:], activation="gelu", stream=stream)
        q.qgemm_w8a8(self.a2, self.s2, *self.w2, self.y2, stream=stream)

    def wanted(self, x):
        self.x.copy_(x)
        self.run()
        torch.cuda.synchronize()
        return self.y2.clone()


@pytest.mark.parametrize("tokens", [1, 16, 48, 200])
def test_graphs(tokens):
    """Captured and replayed on other inputs; two graphs of the same shapes (with scratch of the pool's) at once on two streams."""
    chains = [Chain(tokens, 10), Chain(tokens, 20)]
    inputs = [randn(tokens, 1024, seed=s) for s in range(30, 36)]
    want = [[c.wanted(x) for x in inputs] for c in chains]
    graphs = []
    for c in chains:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in chains]
    torch.cuda.synchronize()
    for i, x in enumerate(inputs):
        got = []
        for c, g, st in zip(chains, graphs, streams):
            with torch.cuda.stream(st):
                c.x.copy_(x)
                c.y2.zero_()
                g.replay()
                g.replay()
                got.append(c.y2.clone())
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(got[k], want[k][i])
    assert q.qgemm_poll_device_error() == 0


@pytest.mark.parametrize("tokens", [3, 40, 260])
def test_streams(tokens):
    """Calls on several streams at once, each with its own buffers; `stream` as an argument and as the current one."""
    chains = [Chain(tokens, 10 * k) for k in range(1, 5)]
    want = [c.wanted(c.x.clone()) for c in chains]
    streams = [torch.cuda.Stream() for _ in chains]
    for c in chains:
        c.y2.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for k, (c, st) in enumerate(zip(chains, streams)):
            if k % 2:
                c.run(stream=st)
            else:
                with torch.cuda.stream(st):
                    c.run()
    torch.cuda.synchronize()
    for c, w in zip(chains, want):
        assert torch.equal(c.y2, w)


def test_order_on_one_stream():
    """Each call sees what the one before it wrote, and what it reads is not overwritten early: buffers reused at once."""
    tokens = 64
    x = [randn(tokens, 4096, seed=s) for s in range(8)]
    w = channels(randn(4096, 4096, seed=9, scale=0.02))
    a, s = torch.empty(tokens, 4096, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")
    y = torch.empty(tokens, 4096, dtype=F, device="cuda")
    want = []
    for v in x:
        q.qgemm_act_quant(v, a, s)
        q.qgemm_w8a8(a, s, *w, y)
        torch.cuda.synchronize()
        want.append(y.clone())
    for _ in range(5):
        got = []
        for v in x:
            q.qgemm_act_quant(v, a, s)
            q.qgemm_w8a8(a, s, *w, y)
            got.append(y.clone())
        for g, t in zip(got, want):
            assert torch.equal(g, t)


def test_example():
    spec = importlib.util.spec_from_file_location("int8_layers", os.path.join(ROOT, "examples", "int8_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    lines = []
    assert m.main(batch=20, steps=6, say=lines.append) < 0.1
    assert len(lines) == 1


@pytest.mark.parametrize("tokens", [4, 40, 300])
def test_operands_written_just_before(tokens):
    """Weights, tokens and scales quantised by the calls right ahead of the product, in buffers that the product before it still
    reads: the product's copies begin early, but not before those calls are done."""
    w = [randn(2048, 1024, seed=s, scale=0.03) for s in range(6)]
    x = [randn(tokens, 1024, seed=10 + s) for s in range(6)]
    codes, scales = torch.empty(2048, 1024, dtype=torch.int8, device="cuda"), torch.empty(2048, device="cuda")
    a, s = torch.empty(tokens, 1024, dtype=torch.int8, device="cuda"), torch.empty(tokens, device="cuda")

    def run(i, c):
        q.qgemm_act_quant(x[i], a, s)
        q.qgemm_act_quant(w[i], codes, scales)
        q.qgemm_w8a8(a, s, codes, scales, c)

    want = []
    for i in range(6):
        c = torch.empty(tokens, 2048, dtype=F, device="cuda")
        run(i, c)
        torch.cuda.synchronize()
        y, size = ref.product(a, s, codes, scales)
        ref.check_product(c, y, size, 1024, 1024 * 127 ** 2)
        want.append(c)
    for _ in range(10):
        got = [torch.empty_like(c) for c in want]
        for i in range(6):
            run(i, got[i])
        for g, t in zip(got, want):
            assert torch.equal(g, t)

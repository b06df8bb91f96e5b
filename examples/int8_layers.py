"""Transformer layers in 8 bits over a paged key-value cache, with random weights: one decode step for a batch of
sequences, captured into a graph and replayed.  Every linear layer is a product of 8-bit integers (qgemm_w8a8); what
stands between them leaves the integers in the same pass: the norm with the residual's addition, the gated activation,
the attention's output.

    python examples/int8_layers.py

Prints the time of a step and checks the last hidden states against the same model in plain torch operations, in 32
bits, with the same (dequantised) weights and activations that are not quantised.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_quantized_tcgen05_gb300 as q  # noqa: E402

HIDDEN, MLP, HQ, HKV, D, LAYERS, PAGE = 1024, 2816, 8, 2, 128, 2, 16
EPS = 1e-5


def channels(w):
    """A weight matrix as integer codes and a scale for each output channel."""
    codes = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    scales = torch.empty(w.shape[0], device=w.device)
    q.qgemm_act_quant(w, codes, scales)
    return codes, scales


class Model:
    def __init__(self, batch, steps, dev, seed=0):
        g = torch.Generator(device=dev).manual_seed(seed)

        def weight(n, k):
            return channels((torch.randn(n, k, generator=g, device=dev) * k ** -0.5).to(torch.float16))

        def gain():
            return 1 + 0.1 * torch.randn(HIDDEN, generator=g, device=dev)

        self.layers = [dict(norm1=gain(), qkv=weight((HQ + 2 * HKV) * D, HIDDEN), out=weight(HIDDEN, HQ * D), norm2=gain(),
                            gate_up=weight(2 * MLP, HIDDEN), down=weight(HIDDEN, MLP),
                            bias=(0.1 * torch.randn((HQ + 2 * HKV) * D, generator=g, device=dev)).to(torch.float16))
                       for _ in range(LAYERS)]
        self.last = gain()
        self.rope = q.qgemm_create_rope(D)
        pages = batch * -(-steps // PAGE)
        k, v = (torch.zeros(LAYERS, pages, HKV, PAGE, D, dtype=torch.float16, device=dev) for _ in "kv")
        self.kv = q.qgemm_create_kv_cache(k, v)
        self.table = torch.full((batch, -(-steps // PAGE)), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        self.seqs = torch.arange(batch, dtype=torch.int32, device=dev)
        self.workspace = q.qgemm_paged_attention_workspace(self.kv, batch, HQ)
        # what a step leaves in its buffers
        f16 = dict(dtype=torch.float16, device=dev)
        self.x, self.h, self.y, self.result = (torch.empty(batch, HIDDEN, **f16) for _ in range(4))
        self.qkv = torch.empty(batch, HQ + 2 * HKV, D, **f16)
        self.attended = torch.empty(batch, HQ * D, **f16)
        self.gate_up = torch.empty(batch, 2 * MLP, **f16)
        self.codes = torch.empty(batch, MLP, dtype=torch.int8, device=dev)
        self.scales = torch.empty(batch, device=dev)

    def step(self):
        """One token for every sequence: self.x -> self.result."""
        q.qgemm_kv_resize(self.kv, self.table, self.lens, self.refs, self.seqs, self.lens + 1)
        positions = self.lens - 1
        hidden = self.codes[:, :HIDDEN]
        queries, keys, values = self.qkv.split([HQ, HKV, HKV], 1)
        gate, up = self.gate_up.split([MLP, MLP], 1)
        self.h.copy_(self.x)
        for i, w in enumerate(self.layers):
            if i == 0:
                q.qgemm_norm_quant(self.h, w["norm1"], hidden, self.scales, eps=EPS)
            else:
                q.qgemm_norm_quant(self.y, w["norm1"], hidden, self.scales, residual=self.h, residual_out=self.h, eps=EPS)
            q.qgemm_w8a8(hidden, self.scales, *w["qkv"], self.qkv.view(len(self.x), -1), bias=w["bias"])
            q.qgemm_kv_append(self.kv, i, keys, values, self.seqs, positions, self.table, rope=self.rope, Q=queries)
            q.qgemm_paged_attention(queries, self.kv, i, self.table, self.lens, self.attended.view(-1, HQ, D), workspace=self.workspace)
            q.qgemm_act_quant(self.attended, hidden, self.scales)
            q.qgemm_w8a8(hidden, self.scales, *w["out"], self.y)
            q.qgemm_norm_quant(self.y, w["norm2"], hidden, self.scales, residual=self.h, residual_out=self.h, eps=EPS)
            q.qgemm_w8a8(hidden, self.scales, *w["gate_up"], self.gate_up)
            q.qgemm_act_quant(gate, self.codes, self.scales, up=up, activation="silu")
            q.qgemm_w8a8(self.codes, self.scales, *w["down"], self.y)
        q.qgemm_norm_quant(self.y, self.last, self.result, residual=self.h, residual_out=self.h, eps=EPS)


def plain(m, inputs):
    """The last hidden states for inputs [steps, batch, HIDDEN], in plain operations."""
    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w

    def linear(x, w, bias=None):
        y = x @ (w[0].float() * w[1][:, None]).T
        return y if bias is None else y + bias.float()

    h = inputs.float()
    steps = len(h)
    angle = torch.arange(steps, device=h.device)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device=h.device) / D)
    cos, sin = angle.cos()[:, None, None], angle.sin()[:, None, None]

    def turned(x):
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)

    later = torch.ones(steps, steps, dtype=torch.bool, device=h.device).triu(1)
    for w in m.layers:
        qkv = linear(norm(h, w["norm1"]), w["qkv"], w["bias"]).unflatten(-1, (-1, D))
        queries, keys, values = qkv.split([HQ, HKV, HKV], 2)
        queries = turned(queries).unflatten(2, (HKV, HQ // HKV))
        score = torch.einsum("sbhgd,tbhd->bhgst", queries, turned(keys)) / math.sqrt(D)
        p = torch.softmax(score.masked_fill(later, -math.inf), -1)
        h = h + linear(torch.einsum("bhgst,tbhd->sbhgd", p, values).flatten(2), w["out"])
        gate, up = linear(norm(h, w["norm2"]), w["gate_up"]).split([MLP, MLP], -1)
        h = h + linear(gate * torch.sigmoid(gate) * up, w["down"])
    return norm(h, m.last)[-1]


def main(batch=40, steps=24, say=print):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(1)
    inputs = torch.randn(steps, batch, HIDDEN, generator=g, device=dev).to(torch.float16)
    m = Model(batch, steps, dev)
    m.x.copy_(inputs[0])
    m.step()                                        # as it is, then captured
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for x in inputs[1:]:
        m.x.copy_(x)
        graph.replay()
    end.record()
    if q.qgemm_poll_device_error():
        raise RuntimeError("a kernel reported an error")
    want = plain(m, inputs)
    off = float((m.result.float() - want).norm() / want.norm())
    say(f"{batch} sequences, {LAYERS} layers of {HIDDEN}: {start.elapsed_time(end) / (steps - 1) * 1e3:.1f} us a step; "
        f"hidden states {100 * off:.2f} % from those without quantised activations")
    return off


if __name__ == "__main__":
    sys.exit(0 if main() < 0.1 else 1)

"""A decode loop over a paged key-value cache, with random weights: prefill of a few prompts of different
lengths, decode steps that grow every sequence by a token, a fork, a freed sequence and a compaction on
the way.  Each layer is int8 projections (qgemm_w8_gemv), rotary positions and the cache's append in one
launch, and attention over the pages; the cache holds E4M3 codes with a scale per 32 elements.

    python examples/decode_serving.py

Prints the time of a step and checks the attention outputs of the last step against a plain softmax over
the keys and values the loop appended.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_quantized_tcgen05_gb300 as q  # noqa: E402
from block_scaled_quantized_tcgen05_gb300 import synth  # noqa: E402

HIDDEN, HQ, HKV, D, PAGE, LAYERS = 1024, 8, 2, 128, 16, 2
SLOTS, MAX_PAGES, PAGES = 8, 16, 96


class Model:
    """LAYERS layers of attention alone: h + W_o attend(W_qkv h)."""

    def __init__(self, dev, seed=0):
        self.dev = dev
        self.weights = []
        for layer in range(LAYERS):
            pair = []
            for n, k, s in (((HQ + 2 * HKV) * D, HIDDEN, 0), (HIDDEN, HQ * D, 1)):
                w = synth.w8_inputs(1, n, k, seed=seed + 10 * layer + s)
                pair.append(q.qgemm_create_tensor(q.INT8, w["w"].to(dev), w["sw"].to(dev)))
            self.weights.append(pair)
        self.rope = q.qgemm_create_rope(D, scaling="by_parts", factor=4.0, original_len=2048)
        shape = (LAYERS, PAGES, HKV, PAGE)
        k, v = (torch.zeros(*shape, D, dtype=torch.uint8, device=dev) for _ in "kv")
        ks, vs = (torch.zeros(*shape, D // 32, dtype=torch.uint8, device=dev) for _ in "kv")
        self.kv = q.qgemm_create_kv_cache(k, v, ks, vs)
        self.table = torch.full((SLOTS, MAX_PAGES), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(SLOTS, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device=dev)
        self.workspace = q.qgemm_paged_attention_workspace(self.kv, SLOTS, HQ)
        self.seen = {}                # (layer, slot) -> [(rotated key, value)], kept for the check alone

    def step(self, h, seqs, keep=None):
        """One token for each of the sequences `seqs` (int32, on the device): h [tokens, HIDDEN] -> the same.  Grows
        them first, so their tokens go to the last position each holds."""
        n = h.shape[0]
        index = seqs.long()
        q.qgemm_kv_resize(self.kv, self.table, self.lens, self.refs, seqs, self.lens[index] + 1)
        positions = self.lens[index] - 1
        outs = []
        for layer, (wqkv, wo) in enumerate(self.weights):
            qkv = torch.empty(n, HQ + 2 * HKV, D, dtype=torch.float16, device=self.dev)
            q.qgemm_w8_gemv(h, wqkv, qkv.view(n, -1))
            queries, keys, values = qkv.split([HQ, HKV, HKV], 1)
            if keep is not None:
                keep(layer, keys, values, positions)
            q.qgemm_kv_append(self.kv, layer, keys, values, seqs, positions, self.table, rope=self.rope, Q=queries)
            o = torch.empty(n, HQ, D, dtype=torch.float16, device=self.dev)
            q.qgemm_paged_attention(queries, self.kv, layer, self.table, self.lens, o, seqs=seqs, workspace=self.workspace)
            y = torch.empty(n, HIDDEN, dtype=torch.float16, device=self.dev)
            q.qgemm_w8_gemv(o.view(n, -1), wo, y)
            outs.append((queries, o))
            h = h + y
        return h, outs


def plain_attention(queries, keys, values):
    s = torch.einsum("hgd,thd->hgt", queries.view(HKV, HQ // HKV, D), keys) / math.sqrt(D)
    return torch.einsum("hgt,thd->hgd", torch.softmax(s, -1), values).reshape(HQ, D)


def in_front(refs):
    """Whether the pages in use are the first ones."""
    used = int((refs > 0).sum())
    return bool((refs[:used] > 0).all())


def main(steps=24, say=print):
    dev = torch.device("cuda:0")
    torch.manual_seed(0)
    m = Model(dev)
    record = {}                       # slot -> per layer, the keys (rotated) and values appended so far

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def keep_for(slots):
        def keep(layer, keys, values, positions):
            turned = keys.contiguous().clone()
            q.qgemm_rope(turned, positions, m.rope)
            for i, s in enumerate(slots):
                record.setdefault(s, [[] for _ in range(LAYERS)])[layer].append((turned[i].float(), values[i].float()))
        return keep

    def run(slots):
        h = torch.randn(len(slots), HIDDEN, device=dev).to(torch.float16)
        return m.step(h, ints(slots), keep_for(slots))

    prompts = {0: 21, 1: 3, 2: 40}
    for t in range(max(prompts.values())):                      # prompts, a token at a time
        run([s for s, n in prompts.items() if t < n])
    live = [0, 1, 2]
    for t in range(steps):
        if t == steps // 3:                                     # two continuations of sequence 0
            q.qgemm_kv_fork(m.kv, m.table, m.lens, m.refs, ints([0, 0]), ints([3, 4]))
            for c in (3, 4):
                record[c] = [list(x) for x in record[0]]
            live += [3, 4]
        if t == steps // 2:                                     # one ends; its pages are taken together
            q.qgemm_kv_resize(m.kv, m.table, m.lens, m.refs, ints([2]))
            if in_front(m.refs):
                raise RuntimeError("the sequence that ended left no holes")
            q.qgemm_kv_compact(m.kv, m.table, m.lens, m.refs)
            if not in_front(m.refs):
                raise RuntimeError("the cache is not compact")
            live.remove(2)
        _, outs = run(live)
    if (word := q.qgemm_poll_device_error()) != 0:
        raise RuntimeError(f"device error word {word:#x}")
    used = int((m.refs > 0).sum())
    if not in_front(m.refs):                                    # free pages are taken lowest first
        raise RuntimeError("the cache is not compact")

    # an E4M3 value is off by 2^-4 of itself at most (and 2^-10 of its block's unit): scores by that of |q| |k|,
    # outputs by that of the weighted |v|; random signs leave a small part of it
    worst = 0.0
    for layer, (queries, o) in enumerate(outs):
        for i, s in enumerate(live):
            keys, values = (torch.stack([x[j] for x in record[s][layer]]) for j in (0, 1))
            want = plain_attention(queries[i].float(), keys, values)
            worst = max(worst, float((o[i].float() - want).norm() / want.norm()))
    if not worst < 0.1:
        raise RuntimeError(f"attention differs from the plain softmax by {worst:.3f}")

    h = torch.randn(len(live), HIDDEN, device=dev).to(torch.float16)
    seqs = ints(live)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    m.step(h, seqs)
    start.record()
    for _ in range(10):
        m.step(h, seqs)
    stop.record()
    torch.cuda.synchronize()
    say(f"{len(live)} sequences of {m.lens[seqs.long()].tolist()} tokens in {used} pages: "
        f"{start.elapsed_time(stop) * 100:.0f} us a step of {LAYERS} layers, attention within {worst:.3f} of a plain softmax")
    return worst


if __name__ == "__main__":
    main()

"""Plain 64-bit restatements of the decode-serving operators, and the tolerances their tests use.

A rounding to a 16-bit type is off by at most half a step, HALF[t] relative to the value.
"""
import math

import numpy as np
import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}      # half the smallest subnormal


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=4.0):
    w = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        w = [x / factor for x in w]
    if scaling == "by_parts":
        keep = [min(1.0, max(0.0, (original_len * x / (2 * math.pi) - low) / (high - low))) for x in w]
        w = [x * (k + (1 - k) / factor) for x, k in zip(w, keep)]
    return torch.tensor(w, dtype=torch.float64)


def rotate(x, pos, rot, interleaved=False, inverse=False, mscale=1.0, **scaling):
    """x [T, H, d] in 64 bits, turned; also the magnitude |a| + |b| each output is formed from."""
    x = x.double()
    angle = pos.double()[:, None] * frequencies(rot, **scaling)
    c, s = (mscale * angle.cos())[:, None], (mscale * angle.sin())[:, None] * (-1 if inverse else 1)
    y, mag = x.clone(), x.abs().clone()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * abs(mscale)
    return y, mag


def rope_tolerance(y, mag, dtype):
    """One rounding of the output, and 2^-21 of what it is formed from: the sine's 2^-23 or so, the
    angle's 2^-24 pi and two fp32 roundings of each product."""
    return HALF[dtype] * (1 + 2.0 ** -8) * y.abs() + 2.0 ** -21 * mag + TINY[dtype]


def e4m3(codes):
    return torch.from_numpy(np.ascontiguousarray(codes.cpu().numpy())).view(torch.float8_e4m3fn).double()


def dequant(codes, scales, dtype):
    """Cached E4M3 rows as the attention takes them: code * 2^(byte - 127), the nearest `dtype` value."""
    d = codes.shape[-1]
    b = scales[..., :d // 32].cpu().double()
    s = torch.where(b == 255, float("nan"), torch.exp2(b - 127))
    x = e4m3(codes) * s.repeat_interleave(32, -1)
    return x.to(dtype).double()


def attend(q, k, v, scale):
    """(o, lse, D, S) of one query row set q [G, d] over k, v [n, d] in 64 bits: D = sum p |v| / sum p and S
    the largest sum of |q k| scale that a score is formed from."""
    q, k, v = q.double(), k.double(), v.double()
    n = k.shape[0]
    if n == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64)
        return z, torch.full((q.shape[0],), -math.inf, dtype=torch.float64), z.clone(), 0.0
    s = q @ k.T * scale
    p = torch.softmax(s, -1)
    size = (q.abs() @ k.abs().T * scale).max().item()
    return p @ v, torch.logsumexp(s, -1), p @ v.abs(), size


def attend_tolerance(o, D, S, n, vmax, dtype):
    """One rounding of the output; P as two 16-bit values (2^-21 or, in bf16, 2^-16 of D) and 2^-39 of the
    largest weight a token; scores summed in fp32 over up to 128 products (16 products of 16 at
    2^-22 of S) and the exponential's argument (2^-23 of S), both sides of the quotient."""
    split = 2.0 ** -20 if dtype == torch.float16 else 2.0 ** -15
    score = (16 * 2.0 ** -22 + 2.0 ** -22) * max(S, 1.0)
    return HALF[dtype] * (1 + 2.0 ** -8) * o.abs() + (split + 2 * score) * D + n * 2.0 ** -38 * vmax + TINY[dtype]


def lse_tolerance(lse, S):
    return 2.0 ** -18 * max(S, 1.0) + 2.0 ** -21 * torch.nan_to_num(lse, neginf=0.0).abs()


class Pages:
    """The page operations on the host, one item after the other."""

    def __init__(self, table, lens, refs, page):
        self.table = [list(r) for r in table]
        self.lens, self.refs, self.page = list(lens), list(refs), page
        self.moves = []          # (src, dst, tokens), in no order that matters

    def of(self, n):
        return -(-n // self.page)

    def shrink(self, s, n):
        for j in range(self.of(n), self.of(self.lens[s])):
            self.refs[self.table[s][j]] -= 1
            self.table[s][j] = -1
        self.lens[s] = n

    def resize(self, seqs, new):
        for s, n in zip(seqs, new):
            if n < self.lens[s]:
                self.shrink(s, n)
        free = [p for p, r in enumerate(self.refs) if r <= 0]
        plan, at, short = [], 0, []
        for s, n in zip(seqs, new):
            need, copy = 0, 0
            if n > self.lens[s]:
                need = self.of(n) - self.of(self.lens[s])
                copy = self.lens[s] % self.page
                if copy and self.refs[self.table[s][self.lens[s] // self.page]] > 1:
                    need += 1
                else:
                    copy = 0
            plan.append((s, n, need, copy, at))
            at += need
        for s, n, need, copy, at in plan:
            if n <= self.lens[s]:
                continue
            if at + need > len(free) and need:
                short.append(s)
                continue
            have, got = self.of(self.lens[s]), free[at:at + need]
            if copy:
                src, dst = self.table[s][have - 1], got.pop(0)
                self.moves.append((src, dst, copy))
                self.refs[src] -= 1
                self.refs[dst] = 1
                self.table[s][have - 1] = dst
            for j, p in enumerate(got):
                self.table[s][have + j] = p
                self.refs[p] = 1
            self.lens[s] = n
        return short

    def fork(self, parents, children):
        for c in children:
            self.shrink(c, 0)
        free = [p for p, r in enumerate(self.refs) if r <= 0]
        at, short = 0, []
        for p, c in zip(parents, children):
            full, tail = divmod(self.lens[p], self.page)
            if tail:
                at += 1
                if at > len(free):
                    short.append(c)
                    continue
            self.table[c][:full] = self.table[p][:full]
            for x in self.table[p][:full]:
                self.refs[x] += 1
            if tail:
                dst = free[at - 1]
                self.table[c][full] = dst
                self.refs[dst] = 1
                self.moves.append((self.table[p][full], dst, tail))
            self.lens[c] = self.lens[p]
        return short

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        holes = [p for p in range(used) if self.refs[p] <= 0]
        movers = [p for p in range(used, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.moves.append((a, b, self.page))
        for s, n in enumerate(self.lens):
            for j in range(self.of(n)):
                self.table[s][j] = to.get(self.table[s][j], self.table[s][j])

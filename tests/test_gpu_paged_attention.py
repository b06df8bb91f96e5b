"""Single-token attention over the paged cache on the GPU against a 64-bit softmax (tests/kv_reference.py
derives the tolerances)."""
import math

import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from block_scaled_quantized_tcgen05_gb300 import build
    build.build()
    q.load_library()
    return torch.device("cuda:0")


class Problem:
    """A cache with sequences of the given lengths in shuffled pages; everything past a length, and
    every unused page, is NaN."""

    def __init__(self, dev, lens, hq, hkv, d, page, dtype, e4m3, order="lphtd", seed=0, size=1.0, spare=2, rows=None):
        self.dev, self.lens, self.hq, self.hkv, self.d, self.page, self.dtype, self.e4m3 = dev, lens, hq, hkv, d, page, dtype, e4m3
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        ids = torch.randperm(pages, generator=g).to(torch.int32)
        self.rows = list(range(B)) if rows is None else rows
        ns = max(self.rows, default=0) + 1
        self.table = torch.full((ns, max(need + [1]) + 1), -1, dtype=torch.int32)
        self.seq_lens = torch.zeros(ns, dtype=torch.int32)
        shape = dict(l=2, p=pages, h=hkv, t=page)
        perm = [c for c in order if c != "d"]
        back = [perm.index(c) for c in "lpht"]

        def plane(inner, dt, fill):
            return torch.full([shape[c] for c in perm] + [inner], fill, dtype=dt).permute(*back, 4)

        if e4m3:
            self.k, self.v = (plane(d, torch.uint8, 0x7F) for _ in "kv")
            self.ks, self.vs = (plane(4, torch.uint8, 255) for _ in "kv")
        else:
            self.k, self.v = (plane(d, dtype, float("nan")) for _ in "kv")
        self.seen = []
        at = 0
        for s, n, m in zip(self.rows, lens, need):
            self.table[s, :m] = ids[at:at + m]
            self.seq_lens[s] = n
            at += m
            t = torch.arange(n)
            pg, off = self.table[s, t // page].long(), t % page
            kv = []
            for name, amp in (("k", size), ("v", 1.0)):
                if e4m3:
                    codes = torch.randint(0, 256, (n, hkv, d), generator=g, dtype=torch.uint8)
                    codes[(codes & 0x7F) == 0x7F] = 0x31
                    b = torch.randint(117, 122, (n, hkv, 4), generator=g, dtype=torch.uint8)
                    getattr(self, name)[1, pg, :, off] = codes
                    getattr(self, name + "s")[1, pg, :, off] = b
                    kv.append(ref.dequant(codes, b, dtype))
                else:
                    x = (amp * torch.randn(n, hkv, d, generator=g)).to(dtype)
                    getattr(self, name)[1, pg, :, off] = x
                    kv.append(x.double())
            self.seen.append(kv)
        self.q = torch.randn(B, hq, d, generator=g).to(dtype)
        self.names = ("k", "v", "ks", "vs") if e4m3 else ("k", "v")

    def upload(self):
        dv = {n: getattr(self, n).to(self.dev) for n in self.names}
        return q.qgemm_create_kv_cache(dv["k"], dv["v"], dv.get("ks"), dv.get("vs"))

    def run(self, scale=None, window=0, workspace=None, lse=True, kv=None):
        kv = kv or self.upload()
        qd = self.q.to(self.dev)
        o = torch.full_like(qd, 9.0)
        l = torch.full((len(self.lens), self.hq), 9.0, device=self.dev) if lse else None
        seqs = torch.tensor(self.rows, dtype=torch.int32, device=self.dev)
        q.qgemm_paged_attention(qd, kv, 1, self.table.to(self.dev), self.seq_lens.to(self.dev), o, seqs=seqs, lse=l,
                                scale=scale, window=window, workspace=workspace)
        return o, l

    def check(self, o, l, scale=None, window=0, drop=None, what=""):
        scale = self.d ** -0.5 if scale is None else scale
        g = self.hq // self.hkv
        for b, n in enumerate(self.lens):
            keep = torch.ones(n, dtype=torch.bool)
            if window and n > window:
                keep[:n - window] = False
            if drop is not None:
                keep &= ~drop(b, torch.arange(n))
            for h in range(self.hkv):
                k, v = (x[keep, h] for x in self.seen[b])
                qs = self.q[b, h * g:(h + 1) * g]
                want, lse, D, S = ref.attend(qs, k, v, scale)
                vmax = float(v.abs().max()) if len(v) else 0.0
                tol = ref.attend_tolerance(want, D, S, len(v), vmax, self.dtype)
                err = (o[b, h * g:(h + 1) * g].cpu().double() - want).abs()
                assert bool((err <= tol).all()), f"{what} b {b} n {n} h {h}: {(err / tol).max().item():.3g} of the tolerance"
                if l is not None:
                    gl = l[b, h * g:(h + 1) * g].cpu().double()
                    if not len(v):
                        assert bool((gl == -math.inf).all())
                    else:
                        e = (gl - lse).abs() / ref.lse_tolerance(lse, S)
                        assert bool((e <= 1).all()), f"{what} lse {e.max().item():.3g} of the tolerance"


def _clean(word=0):
    assert q.qgemm_poll_device_error() == word


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d,page,order", [
    ([1], 1, 1, 128, 16, "lphtd"),
    ([0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 255, 256, 257], 8, 2, 128, 16, "lphtd"),
    ([500, 0, 77, 1000], 8, 8, 64, 24, "lpthd"),                      # one query head a key-value head
    ([300, 5], 28, 4, 128, 7, "plhtd"),                               # seven: an odd group
    ([260, 64, 1], 9, 1, 64, 1, "lphtd"),                             # nine; pages of one token
    ([700, 33], 32, 2, 128, 100, "lpthd"),                            # sixteen
    ([400, 129], 40, 2, 64, 32, "lphtd"),                             # twenty: two units a head
    ([90], 33, 1, 128, 64, "lphtd"),                                  # thirty-three: three units
])
def test_attention_matches(dev, dtype, e4m3, lens, hq, hkv, d, page, order):
    p = Problem(dev, lens, hq, hkv, d, page, dtype, e4m3, order, seed=len(lens) + hq, size=2.0)
    o, l = p.run()
    _clean()
    p.check(o, l)
    o2, l2 = p.run()
    assert torch.equal(o, o2) and torch.equal(l, l2)                  # repeatable bit for bit


@pytest.mark.parametrize("e4m3", [False, True])
def test_one_sequence_over_many_ctas(dev, e4m3):
    """One key-value head, 40000 tokens: the unit is cut by every range boundary and merged."""
    p = Problem(dev, [40000], 4, 1, 128, 48, torch.float16, e4m3, seed=9, size=3.0)
    kv = p.upload()
    o, l = p.run(kv=kv)
    _clean()
    p.check(o, l)
    for _ in range(3):
        o2, l2 = p.run(kv=kv)
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_ragged_batch_and_row_selection(dev):
    """Lengths from none to thousands; table rows picked out of order, unused rows between them."""
    lens = [0, 3000, 1, 0, 640, 128, 2049, 17, 0, 5000, 1, 90, 511, 512, 513, 0]
    rows = [(7 * i + 3) % 19 for i in range(len(lens))]
    p = Problem(dev, lens, 16, 4, 128, 16, torch.bfloat16, False, seed=4, rows=rows)
    o, l = p.run()
    _clean()
    p.check(o, l)
    o, l = p.run(lse=False)
    _clean()
    p.check(o, None)


@pytest.mark.parametrize("e4m3,dtype", [(False, torch.float16), (True, torch.bfloat16)])
@pytest.mark.parametrize("window", [1, 16, 100, 129, 4096])
def test_window(dev, e4m3, dtype, window):
    p = Problem(dev, [0, 1, 99, 100, 101, 1000, 300], 6, 2, 128, 24, dtype, e4m3, seed=window)
    o, l = p.run(window=window)
    _clean()
    p.check(o, l, window=window)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 4.0])
def test_scales_from_flat_to_one_hot(dev, scale):
    p = Problem(dev, [1500, 200], 8, 1, 64, 16, torch.float16, False, seed=11, size=2.0)
    o, l = p.run(scale=scale)
    _clean()
    p.check(o, l, scale=scale)


def test_rising_maximum_and_small_weights(dev):
    """Keys whose score grows along the sequence raise the running maximum at every step; then one token of
    weight 1 among many of 2^-25, whose sum still counts."""
    p = Problem(dev, [2000], 1, 1, 128, 16, torch.float16, False, seed=12)
    t = torch.arange(2000)
    pg, off = p.table[0, t // 16].long(), t % 16
    p.q[:] = 1.0
    k = (t.float() / 100).to(torch.float16)[:, None, None].expand(-1, 1, 128)
    p.k[1, pg, :, off] = k
    p.seen[0][0] = k.double()
    o, l = p.run()
    p.check(o, l, what="rising")
    k = torch.zeros(2000, 1, 128, dtype=torch.float16)
    k[777] = 25 * math.log(2) / 128 * 128 ** 0.5                     # its score stands 25 ln 2 above
    v = torch.ones(2000, 1, 128, dtype=torch.float16)
    v[777] = 0.0
    p.k[1, pg, :, off], p.v[1, pg, :, off] = k, v
    p.seen[0] = [k.double(), v.double()]
    o, l = p.run()
    p.check(o, l, what="small weights")
    assert float(o.float().min()) > 0
    _clean()


def test_large_values(dev):
    """Values at the end of fp16's range: the weighted sum stays finite."""
    p = Problem(dev, [300], 2, 1, 64, 16, torch.float16, False, seed=13)
    t = torch.arange(300)
    v = torch.full((300, 1, 64), 60000.0, dtype=torch.float16)
    p.v[1, p.table[0, t // 16].long(), :, t % 16] = v
    p.seen[0][1] = v.double()
    o, l = p.run()
    _clean()
    p.check(o, l)


def test_special_values_reach_the_output(dev):
    """A NaN or infinity among the seen keys or values shows in that head's output, and in no other."""
    for e4m3 in (False, True):
        p = Problem(dev, [100, 100], 4, 2, 128, 16, torch.float16, e4m3, seed=14)
        pg, off = int(p.table[0, 3]), 2                               # token 50 of the first sequence
        if e4m3:
            p.v[1, pg, 1, off, 7] = 0x7F
            p.ks[1, pg, 0, off, 2] = 255
        else:
            p.v[1, pg, 1, off, 7] = float("inf")
            p.k[1, pg, 0, off, 64] = float("nan")
        o, l = p.run()
        _clean()
        o = o.cpu().float()
        assert bool(o[0, :2].isnan().all()) and bool(l[0, :2].isnan().all())
        bad = ~o[0, 2:].isfinite()
        assert bool(bad[:, 7].all()) and int(bad.sum()) == 2
        assert bool(o[1].isfinite().all())
        if not e4m3:
            assert bool((o[0, 2:, 7] == float("inf")).all())


def test_infinite_value_of_a_small_weight(dev):
    """A weight far below what 16 bits hold is still not zero: times infinity it is infinity."""
    for dtype in (torch.float16, torch.bfloat16):
        p = Problem(dev, [100], 1, 1, 128, 16, dtype, False, seed=21)
        p.k[1, p.table[0, 0], 0, 0] = (4 * p.q[0, 0].float()).to(dtype)      # e^45 times the others' weights
        pg, off = int(p.table[0, 3]), 2                                # token 50
        p.v[1, pg, 0, off, 7], p.v[1, pg, 0, off, 9] = float("inf"), float("-inf")
        o, l = p.run()
        _clean()
        o = o.cpu().float()[0, 0]
        assert o[7] == float("inf") and o[9] == float("-inf")
        assert bool(l.isfinite().all()) and int((~o.isfinite()).sum()) == 2


def test_every_scale_byte(dev):
    """UE8M0 bytes far outside the halves: values are the nearest half (bfloat16) to the product, infinity
    where it overflows."""
    for dtype in (torch.float16, torch.bfloat16):
        for lo, hi in ((90, 150), (0, 40), (95, 108), (140, 144)):
            p = Problem(dev, [200], 2, 1, 128, 16, dtype, True, seed=lo)
            g = torch.Generator().manual_seed(lo)
            t = torch.arange(200)
            pg, off = p.table[0, t // 16].long(), t % 16
            codes = p.v[1, pg, :, off].clone()
            codes[(codes & 0x78) == 0x78] = 0x30                      # below 256: overflow by the scale alone
            if lo == 140:                                              # E4M3 subnormals stay finite halves
                codes &= 0x87
            b = torch.randint(lo, hi, (200, 1, 4), generator=g, dtype=torch.uint8)
            if dtype == torch.float16 and lo != 140:
                b.clamp_(max=127)
            p.v[1, pg, :, off], p.vs[1, pg, :, off] = codes, b
            p.seen[0][1] = ref.dequant(codes, b, dtype)
            assert bool(p.seen[0][1].isfinite().all())
            o, l = p.run()
            _clean()
            p.check(o, l, what=f"bytes {lo}..{hi}")


@pytest.mark.parametrize("d,hq,hkv", [(128, 5, 1), (64, 24, 2)])
@pytest.mark.parametrize("power,byte", [(0, 119), (60, 59), (-60, 179), (-110, 229), (100, 19), (30, 119)])
def test_bf16_queries_of_any_size_meet_e4m3_keys(dev, d, hq, hkv, power, byte):
    """Query rows of very different sizes, wide ranges inside a row, keys whose scales make up for them."""
    p = Problem(dev, [200, 3], hq, hkv, d, 16, torch.bfloat16, True, seed=power % 97)
    g = torch.Generator().manual_seed(d + power % 97)
    p.q = (p.q.float() * 2.0 ** (power + torch.randint(-12, 1, p.q.shape, generator=g).float())).to(torch.bfloat16)
    p.q[:, 0] = 0.0
    if power == 30:                                       # sizes only a power of two apart from a row's own keys
        p.q = (p.q.float() * 2.0 ** -30).to(torch.bfloat16)
        p.q[0, 1] *= 2.0 ** -40
        p.q[1, 2, 5] = 2.0 ** -126
    for b, n in enumerate(p.lens):
        t = torch.arange(n)
        pg, off = p.table[p.rows[b], t // 16].long(), t % 16
        sc = torch.randint(byte - 2, byte + 3, (n, hkv, 4), generator=g, dtype=torch.uint8)
        p.ks[1, pg, :, off] = sc
        p.seen[b][0] = ref.dequant(p.k[1, pg, :, off], sc, torch.bfloat16)
    o, l = p.run(scale=1.0)
    _clean()
    p.check(o, l, scale=1.0)


def test_bad_pages_and_lengths_are_skipped(dev):
    """Table entries that name no page: their tokens are absent; a length past the table row ends with the
    row; a sequence number out of range is an empty sequence.  The error word says so each time."""
    p = Problem(dev, [100, 64], 4, 2, 128, 16, torch.float16, False, seed=15)
    good = p.table.clone()
    p.table[0, 2], p.table[0, 5] = -1, 10 ** 6
    o, l = p.run()
    _clean(64)
    p.check(o, l, drop=lambda b, t: ((t // 16 == 2) | (t // 16 == 5)) if b == 0 else torch.zeros(len(t), dtype=torch.bool))
    p.table = good.clone()
    p.table[0, :] = -1
    o, l = p.run()
    _clean(64)
    p.check(o, l, drop=lambda b, t: torch.full((len(t),), b == 0))
    p.table = good[:, :4].clone()                                     # rows of 64 tokens
    o, l = p.run()
    _clean(64)
    p.check(o, l, drop=lambda b, t: t >= 64)
    p.table = good
    p.rows = [0, 7]
    o, l = p.run()
    _clean(64)
    p.check(o, l, drop=lambda b, t: torch.full((len(t),), b == 1))
    p.rows, p.seq_lens[0] = [0, 1], -5
    o, l = p.run()
    _clean(64)
    p.check(o, l, drop=lambda b, t: torch.full((len(t),), b == 0))


def test_workspace_serves_other_batches(dev):
    """One workspace, calls of several batches and head counts one after another."""
    big = Problem(dev, [900] * 6, 32, 4, 128, 16, torch.float16, False, seed=16)
    small = Problem(dev, [5000, 20], 8, 2, 128, 16, torch.float16, True, seed=17)
    kb, ks = big.upload(), small.upload()
    ws = q.qgemm_paged_attention_workspace(kb, 6, 32)
    want = [big.run(kv=kb), small.run(kv=ks)]
    for _ in range(3):
        for p, k, (wo, wl) in ((big, kb, want[0]), (small, ks, want[1])):
            o, l = p.run(kv=k, workspace=ws)
            assert torch.equal(o, wo) and torch.equal(l, wl)
    _clean()


def test_strided_queries_and_outputs(dev):
    """Queries inside a fused projection's rows, outputs with heads outside sequences: only O is written."""
    p = Problem(dev, [300, 40, 7], 8, 2, 128, 16, torch.float16, False, seed=18)
    kv = p.upload()
    want, _ = p.run(kv=kv)
    fused = torch.randn(3, 12, 128, device=dev).to(torch.float16)
    fused[:, 2:10] = p.q.to(dev)
    buf = torch.full((8, 3, 136), 5.0, dtype=torch.float16, device=dev)
    o = buf[:, :, :128].transpose(0, 1)
    q.qgemm_paged_attention(fused[:, 2:10], kv, 1, p.table.to(dev), p.seq_lens.to(dev), o)
    _clean()
    assert torch.equal(o, want) and bool((buf[:, :, 128:] == 5.0).all())


def test_offsets_past_32_bits(dev):
    """A cache of more than 2^32 bytes: pages at its end."""
    pages, page, h, d = 1100, 64, 256, 128                              # 4.6 GB a plane
    k = torch.empty(1, pages, h, page, d, dtype=torch.float16, device=dev)
    v = torch.empty_like(k)
    kv = q.qgemm_create_kv_cache(k, v)
    ids = [pages - 1, pages - 3, 1]
    n = 150
    for x in ids:
        k[0, x].normal_()
        v[0, x].normal_()
    table = torch.tensor([ids], dtype=torch.int32, device=dev)
    qd = torch.randn(1, h, d, device=dev).to(torch.float16)
    o = torch.empty_like(qd)
    q.qgemm_paged_attention(qd, kv, 0, table, torch.tensor([n], dtype=torch.int32, device=dev), o)
    _clean()
    for head in (0, 100, 255):
        ks, vs = (torch.cat([x[0, i, head] for i in ids])[:n].cpu() for x in (k, v))
        want, _, D, S = ref.attend(qd[0, head:head + 1].cpu(), ks, vs, d ** -0.5)
        tol = ref.attend_tolerance(want, D, S, n, float(vs.abs().max()), torch.float16)
        assert bool(((o[0, head:head + 1].cpu().double() - want).abs() <= tol).all())


def test_streams_and_graph(dev):
    """Calls on side streams with workspaces of their own give the serial bits; a captured call serves other
    lengths, written into its buffers, without another capture."""
    ps = [Problem(dev, [1000 + 300 * i, 5, 0, 2000], 16, 4, 128, 32, torch.float16, bool(i % 2), seed=20 + i) for i in range(3)]
    kvs = [p.upload() for p in ps]
    want = [p.run(kv=kv) for p, kv in zip(ps, kvs)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    args = []
    for p, kv in zip(ps, kvs):
        args.append((p.q.to(dev), kv, 1, p.table.to(dev), p.seq_lens.to(dev), torch.empty_like(p.q, device=dev)))
    ws = [q.qgemm_paged_attention_workspace(kv, 4, 16) for kv in kvs]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, w, s in zip(args, ws, streams):
            q.qgemm_paged_attention(*a, workspace=w, stream=s)
    torch.cuda.synchronize()
    for a, (o, _) in zip(args, want):
        assert torch.equal(a[5], o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qgemm_paged_attention(*args[0], workspace=ws[0])
    p = ps[0]
    args[0][4].copy_(torch.tensor([700, 2, 0, 1999], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    p.lens = [700, 2, 0, 1999]
    p.seen = [[x[:n] for x in kv] for kv, n in zip(p.seen, p.lens)]
    p.check(args[0][5], None)
    _clean()

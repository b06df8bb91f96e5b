"""Page operations of the paged cache on the GPU against a host restatement (tests/kv_reference.py): tables,
lengths and counts are equal, and so is every byte of the cache."""
import random

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


class State:
    def __init__(self, dev, slots, max_pages, pages, page, heads=2, layers=3, d=64, e4m3=False, order="lphtd", seed=0):
        g = torch.Generator(device=dev).manual_seed(seed)
        shape = dict(l=layers, p=pages, h=heads, t=page)
        perm = [c for c in order if c != "d"]
        back = [perm.index(c) for c in "lpht"]

        def plane(inner):
            return torch.randint(0, 256, [shape[c] for c in perm] + [inner], generator=g, dtype=torch.uint8, device=dev).permute(*back, 4)

        if e4m3:
            self.data = [plane(d), plane(d), plane(4), plane(4)]
            self.kv = q.qgemm_create_kv_cache(*self.data)
        else:
            self.data = [plane(2 * d), plane(2 * d)]
            self.kv = q.qgemm_create_kv_cache(*(x.view(torch.float16) for x in self.data))
        self.dev, self.page = dev, page
        self.table = torch.full((slots, max_pages), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(slots, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        self.host = ref.Pages(self.table.tolist(), self.lens.tolist(), self.refs.tolist(), page)

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.dev)

    def before(self):
        self.host.moves = []
        self.old = [x.clone() for x in self.data]

    def same(self, what=""):
        """The device's state is the host's, and the data moved as it says."""
        assert self.table.tolist() == self.host.table, what
        assert self.lens.tolist() == self.host.lens, what
        assert self.refs.tolist() == self.host.refs, what
        for now, old in zip(self.data, self.old):
            want = old.clone()
            for a, b, n in self.host.moves:
                want[:, b, :, :n] = old[:, a, :, :n]
            assert torch.equal(now, want), what

    def resize(self, seqs, new, error=0):
        self.before()
        short = self.host.resize(seqs, new)
        q.qgemm_kv_resize(self.kv, self.table, self.lens, self.refs, self.ints(seqs), self.ints(new))
        assert q.qgemm_poll_device_error() == (128 if short else 0) | error
        self.same(f"resize {seqs} {new}")

    def fork(self, parents, children):
        self.before()
        short = self.host.fork(parents, children)
        q.qgemm_kv_fork(self.kv, self.table, self.lens, self.refs, self.ints(parents), self.ints(children))
        assert q.qgemm_poll_device_error() == (128 if short else 0)
        self.same(f"fork {parents} {children}")

    def compact(self):
        self.before()
        self.host.compact()
        q.qgemm_kv_compact(self.kv, self.table, self.lens, self.refs)
        assert q.qgemm_poll_device_error() == 0
        self.same("compact")


@pytest.mark.parametrize("e4m3,d,page,order", [(False, 64, 8, "lphtd"), (True, 128, 16, "plhtd"), (False, 128, 5, "lpthd"),
                                               (True, 64, 1, "lphtd"), (True, 64, 24, "lpthd")])
def test_a_random_life(dev, e4m3, d, page, order):
    """Growing, truncating, freeing, forking and compacting in random order, pages sometimes short."""
    rng = random.Random(page)
    s = State(dev, 12, 9, 60, page, e4m3=e4m3, d=d, order=order, seed=page)
    cap = 9 * page
    for _ in range(60):
        op = rng.random()
        if op < 0.6:
            seqs = rng.sample(range(12), rng.randint(1, 8))
            s.resize(seqs, [rng.choice([0, min(cap, s.host.lens[x] + 1), rng.randint(0, cap), cap]) for x in seqs])
        elif op < 0.85:
            who = rng.sample(range(12), 6)
            k = rng.randint(1, 4)
            s.fork([rng.choice(who[:2]) for _ in range(k)], who[2:2 + k])
        else:
            s.compact()


def test_copy_on_write_after_truncation(dev):
    """A truncated sequence whose last page is shared gets a page of its own before it grows."""
    s = State(dev, 4, 4, 12, 8)
    s.resize([0], [24])
    s.fork([0, 0], [1, 2])                       # whole pages: shared by three
    s.resize([1, 2], [20, 20])                   # into a shared page
    s.resize([1], [21])
    s.resize([2, 0], [25, 32])
    assert s.host.refs.count(1) > 0
    s.resize([0, 1, 2], [0, 0, 0])
    assert all(r == 0 for r in s.host.refs)


def test_free_without_lengths(dev):
    s = State(dev, 3, 4, 12, 8)
    s.resize([0, 1, 2], [30, 8, 1])
    s.before()
    s.host.resize([2, 0], [0, 0])
    q.qgemm_kv_resize(s.kv, s.table, s.lens, s.refs, s.ints([2, 0]))
    assert q.qgemm_poll_device_error() == 0
    s.same()


def test_many_items_and_pages(dev):
    """More sequences than the bookkeeping block has threads, counts past one scan, then a compaction of all."""
    n, pages = 1500, 20000
    s = State(dev, 2 * n, 12, pages, 2, heads=1, layers=1, d=64, seed=3)
    rng = random.Random(4)
    s.resize(list(range(n)), [rng.randint(0, 24) for _ in range(n)])
    s.resize(rng.sample(range(n), 700), [0] * 700)
    s.fork(rng.sample(range(n), 900), rng.sample(range(n, 2 * n), 900))
    s.compact()
    s.resize(list(range(n)), [24] * n)
    s.resize(list(range(0, n, 2)), [0] * (n // 2))
    s.compact()
    s.compact()                                  # already compact: nothing moves
    assert s.host.moves == []


def test_copy_pages(dev):
    s = State(dev, 1, 1, 40, 24, e4m3=True, d=128, heads=3)
    s.before()
    src, dst = [3, 3, 7, 39], [0, 20, 21, 5]
    s.host.moves = [(a, b, 24) for a, b in zip(src, dst)]
    q.qgemm_kv_copy_pages(s.kv, s.ints(src), s.ints(dst))
    assert q.qgemm_poll_device_error() == 0
    s.same()
    s.before()
    s.host.moves = [(4, 6, 24)]
    q.qgemm_kv_copy_pages(s.kv, s.ints([40, -1, 2, 4, 1]), s.ints([8, 9, 40, 6, -7]))
    assert q.qgemm_poll_device_error() == 64
    s.same()


def test_bad_indices_are_skipped(dev):
    s = State(dev, 4, 3, 12, 8)
    s.resize([0, 1], [17, 9])
    s.before()
    s.host.resize([1], [24])
    q.qgemm_kv_resize(s.kv, s.table, s.lens, s.refs, s.ints([4, -1, 0, 1, 2]), s.ints([8, 8, 25, 24, -1]))
    assert q.qgemm_poll_device_error() == 64
    s.same("resize")
    s.before()
    s.host.fork([0], [3])
    q.qgemm_kv_fork(s.kv, s.table, s.lens, s.refs, s.ints([9, 0, 1]), s.ints([2, 3, -2]))
    assert q.qgemm_poll_device_error() == 64
    s.same("fork")
    # a table entry out of range: skipped, counts and pages stay as they are
    s.table[0, 1] = 500
    refs = s.refs.clone()
    data = [x.clone() for x in s.data]
    q.qgemm_kv_resize(s.kv, s.table, s.lens, s.refs, s.ints([0]), s.ints([0]))
    assert q.qgemm_poll_device_error() == 64
    assert int((refs - s.refs).sum()) == 2 and all(torch.equal(a, b) for a, b in zip(s.data, data))


def test_on_a_side_stream_and_in_a_graph(dev):
    """A captured decode step grows every sequence by a token each time it is replayed."""
    s = State(dev, 4, 6, 30, 4)
    s.resize([0, 1, 2, 3], [3, 4, 0, 9])
    side = torch.cuda.Stream()
    seqs, new = s.ints([0, 1, 2, 3]), s.lens + 1
    side.wait_stream(torch.cuda.current_stream())
    s.before()
    s.host.resize([0, 1, 2, 3], [4, 5, 1, 10])
    q.qgemm_kv_resize(s.kv, s.table, s.lens, s.refs, seqs, new, stream=side)
    side.synchronize()
    s.same("side stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new.copy_(s.lens + 1)
        q.qgemm_kv_resize(s.kv, s.table, s.lens, s.refs, seqs, new)
    for _ in range(7):
        s.before()
        s.host.resize([0, 1, 2, 3], [n + 1 for n in s.host.lens])
        g.replay()
        torch.cuda.synchronize()
        s.same("graph")

"""Forking and growing a sequence whose last, partly filled page is a table entry that names no page: the entry is
reported and kept, so the tokens on it stay absent, and nothing is taken or copied for it."""
import random

import pytest

import block_scaled_quantized_tcgen05_gb300 as q
from tests.test_gpu_kv_pages import State, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def spoil(s, seq, j, entry):
    """The host's page is forgotten as well: its count stays."""
    s.table[seq, j] = entry
    s.host.table[seq][j] = entry


@pytest.mark.parametrize("entry", [-1, 500])
def test_fork_keeps_a_bad_last_entry(dev, entry):  # noqa: F811
    s = State(dev, 6, 3, 12, 8)
    s.resize([0, 3], [13, 9])
    spoil(s, 0, 1, entry)
    s.before()
    s.host.fork([3], [2])                        # the good one, between two bad ones: takes the lowest free page
    for c in (1, 4):
        s.host.table[c] = [s.host.table[0][0], entry, -1]
        s.host.refs[s.host.table[0][0]] += 1
        s.host.lens[c] = 13
    q.qgemm_kv_fork(s.kv, s.table, s.lens, s.refs, s.ints([0, 3, 0]), s.ints([1, 2, 4]))
    assert q.qgemm_poll_device_error() == 64
    s.same("fork")
    s.before()                                   # the children go again: the good page is given back
    s.host.refs[s.host.table[0][0]] -= 2
    for c in (1, 4):
        s.host.table[c], s.host.lens[c] = [-1, -1, -1], 0
    q.qgemm_kv_resize(s.kv, s.table, s.lens, s.refs, s.ints([1, 4]))
    assert q.qgemm_poll_device_error() == 64
    s.same("free")


def test_fork_of_many_with_bad_last_entries(dev):  # noqa: F811
    """More items than the bookkeeping keeps in shared memory."""
    n = 1300
    s = State(dev, 2 * n, 3, 6000, 4, heads=1, layers=1, seed=5)
    rng = random.Random(6)
    s.resize(list(range(n)), [rng.randint(1, 11) for _ in range(n)])
    bad = [x for x in rng.sample(range(n), 60) + [n - 1, n - 2] if s.host.lens[x] % 4]
    for x in bad:
        spoil(s, x, s.host.lens[x] // 4, 10 ** 6)
    s.before()
    good = [x for x in range(n) if x not in set(bad)]
    s.host.fork(good, [n + x for x in good])
    for x in bad:
        full = s.host.lens[x] // 4
        for j in range(full):
            s.host.refs[s.host.table[x][j]] += 1
        s.host.table[n + x], s.host.lens[n + x] = list(s.host.table[x]), s.host.lens[x]
    q.qgemm_kv_fork(s.kv, s.table, s.lens, s.refs, s.ints(list(range(n))), s.ints(list(range(n, 2 * n))))
    assert q.qgemm_poll_device_error() == 64
    s.same("fork")


@pytest.mark.parametrize("entry", [-7, 12])
def test_growth_past_a_bad_last_entry_is_reported(dev, entry):  # noqa: F811
    s = State(dev, 3, 5, 12, 8)
    s.resize([0, 1], [13, 3])
    spoil(s, 0, 1, entry)
    for new in (14, 30):                         # inside the page; into new ones
        s.before()
        have = s.host.lens[0]
        free = [p for p, r in enumerate(s.host.refs) if r <= 0]
        for j in range(s.host.of(have), s.host.of(new)):
            s.host.table[0][j] = free.pop(0)
            s.host.refs[s.host.table[0][j]] = 1
        s.host.lens[0] = new
        q.qgemm_kv_resize(s.kv, s.table, s.lens, s.refs, s.ints([0]), s.ints([new]))
        assert q.qgemm_poll_device_error() == 64
        s.same(f"grow to {new}")

"""Host-side checks of the decode-serving calls (no GPU): refusals with their documented status before
anything touches the device, the index arithmetic the kernels run (compiled for the CPU from the
same header), and the test references against one another."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from block_scaled_quantized_tcgen05_gb300 import build as qbuild
from tests import kv_reference as ref

A = 0x7F0000000000           # fake 256-byte aligned device addresses, never dereferenced on the host
B_ = 0x7E0000000000
INVALID, SHAPE, MISALIGNED, DTYPE, CUDA = 1, 2, 3, 4, 5
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.load_library()


def _cache(lib, dtype=q.F16, layers=2, pages=8, heads=4, page=16, d=128, k=A, v=B_, st=None, ks=None, vs=None, sst=None):
    row = d if dtype == q.E4M3 else 2 * d
    st = st or (pages * heads * page * row, heads * page * row, page * row, row)
    if dtype == q.E4M3 and sst is None:
        sst = (pages * heads * page * 4, heads * page * 4, page * 4, 4)
        ks, vs = ks or A + 0x1000, vs or B_ + 0x1000
    out = ctypes.c_void_p()
    status = lib.qgemm_create_kv_cache(ctypes.byref(out), dtype, layers, pages, heads, page, d, P(k), P(v),
                                       (ctypes.c_int64 * 4)(*st), P(ks), P(vs),
                                       None if sst is None else (ctypes.c_int64 * 4)(*sst))
    assert (status == 0) == bool(out.value)
    return status, out


@pytest.mark.parametrize("change,status", [
    (dict(), 0), (dict(dtype=q.E4M3), 0), (dict(dtype=q.BF16, d=64), 0),
    (dict(dtype=q.INT8), DTYPE), (dict(d=96), SHAPE), (dict(pages=0, st=(1, 1, 1, 1)), INVALID),
    (dict(layers=0, st=(1, 1, 1, 1)), INVALID), (dict(k=0), INVALID), (dict(v=A), INVALID),
    (dict(k=A + 8), MISALIGNED), (dict(st=(131072, 16384, 4096, 264)), MISALIGNED),
    (dict(st=(131072, 16384, 4096, 128)), INVALID),              # tokens overlap
    (dict(st=(131072, 16384, 4080, 256)), INVALID),              # heads overlap
    (dict(st=(65536, 16384, 4096, 256)), INVALID),               # layers overlap
    (dict(st=(131072, 16384, 256, 1024)), 0),                    # tokens outside heads
    (dict(st=(32768, 32768, 4096, 256)), INVALID),               # pages and layers coincide
    (dict(st=(16384, 32768, 4096, 256)), 0),                     # layers inside pages
    (dict(layers=4096, heads=1024, page=512, pages=1, st=(1 << 27, 1 << 40, 1 << 17, 256)), SHAPE),   # 2^31 rows a page
    (dict(ks=A, vs=B_), DTYPE), (dict(dtype=q.E4M3, sst=(512, 64, 16, 2), ks=A, vs=B_), MISALIGNED),
    (dict(dtype=q.E4M3, sst=(2048, 256, 64, 4), ks=A + 2, vs=B_), MISALIGNED),
    (dict(dtype=q.E4M3, sst=(2048, 256, 32, 4), ks=A, vs=B_), INVALID),
    (dict(dtype=q.E4M3, sst=(2048, 256, 64, 4), ks=None, vs=B_), INVALID),
])
def test_cache_view_checks(lib, change, status):
    got, handle = _cache(lib, **change)
    assert got == status, lib.qgemm_last_error_message()
    lib.qgemm_destroy_kv_cache(handle)


@pytest.mark.parametrize("args,status", [
    ((128, 0, 1e4, 0, 1.0, 0.0, 1.0, 4.0, 1.0), 0), ((2, 1, 1e4, 1, 4.0, 0.0, 1.0, 4.0, 1.0), 0),
    ((64, 0, 5e5, 2, 8.0, 8192.0, 1.0, 4.0, 1.1), 0),
    ((0, 0, 1e4, 0, 1.0, 0.0, 1.0, 4.0, 1.0), INVALID), ((7, 0, 1e4, 0, 1.0, 0.0, 1.0, 4.0, 1.0), INVALID),
    ((258, 0, 1e4, 0, 1.0, 0.0, 1.0, 4.0, 1.0), SHAPE), ((64, 2, 1e4, 0, 1.0, 0.0, 1.0, 4.0, 1.0), INVALID),
    ((64, 0, 0.0, 0, 1.0, 0.0, 1.0, 4.0, 1.0), INVALID), ((64, 0, 1e4, 3, 1.0, 0.0, 1.0, 4.0, 1.0), INVALID),
    ((64, 0, 1e4, 1, 0.0, 0.0, 1.0, 4.0, 1.0), INVALID), ((64, 0, 1e4, 2, 2.0, 0.0, 1.0, 4.0, 1.0), INVALID),
    ((64, 0, 1e4, 2, 2.0, 8192.0, 4.0, 4.0, 1.0), INVALID),
    ((64, 0, 1e4, 0, 1.0, 0.0, 1.0, 4.0, float("nan")), INVALID),
])
def test_rope_handle_checks(lib, args, status):
    out = ctypes.c_void_p()
    assert lib.qgemm_create_rope(ctypes.byref(out), *args) == status, lib.qgemm_last_error_message()
    assert bool(out.value) == (status == 0)
    lib.qgemm_destroy_rope(out)


def _rope(lib, rot=64):
    out = ctypes.c_void_p()
    assert lib.qgemm_create_rope(ctypes.byref(out), rot, 0, 1e4, 0, 1.0, 0.0, 1.0, 4.0, 1.0) == 0
    return out


@pytest.mark.parametrize("change,status", [
    (dict(), CUDA),                      # all in order: only the missing GPU stops it here
    (dict(T=0, X=0), 0), (dict(heads=0), 0), (dict(dtype=q.E4M3), DTYPE), (dict(X=0), INVALID), (dict(Y=0), INVALID),
    (dict(pos=0), INVALID), (dict(pos=A + 2), MISALIGNED), (dict(X=A + 1), MISALIGNED), (dict(d=48), SHAPE),
    (dict(d=264), SHAPE), (dict(T=-1), INVALID), (dict(rope=0), INVALID), (dict(inverse=2), INVALID),
    (dict(yt=64), INVALID), (dict(yh=64), INVALID), (dict(xt=-8), INVALID), (dict(T=1 << 31), SHAPE),
])
def test_rope_refusals(lib, change, status):
    if status == CUDA and torch.cuda.is_available():
        pytest.skip("would launch")
    a = dict(X=A, xt=1024, xh=128, Y=B_, yt=1024, yh=128, dtype=q.F16, T=16, heads=8, d=128, pos=A, rope=1, inverse=0)
    a.update(change)
    rope = _rope(lib)
    got = lib.qgemm_rope(P(a["X"]), a["xt"], a["xh"], P(a["Y"]), a["yt"], a["yh"], a["dtype"], a["T"], a["heads"],
                         a["d"], P(a["pos"]), rope if a["rope"] else None, a["inverse"], None)
    assert got == status, lib.qgemm_last_error_message()
    lib.qgemm_destroy_rope(rope)


@pytest.mark.parametrize("change,status", [
    (dict(), CUDA), (dict(T=0, K=0), 0), (dict(kv=0), INVALID), (dict(layer=2), INVALID), (dict(layer=-1), INVALID),
    (dict(dtype=q.BF16), DTYPE), (dict(dtype=q.E4M3), DTYPE), (dict(K=0), INVALID), (dict(V=A + 1), MISALIGNED),
    (dict(seqs=0), INVALID), (dict(pos=A + 1), MISALIGNED), (dict(table=0), INVALID), (dict(ts=4), INVALID),
    (dict(table=A + 2), MISALIGNED), (dict(mp=1 << 28), SHAPE), (dict(ms=-1), INVALID), (dict(Q=0), INVALID),
    (dict(Qo=0), INVALID), (dict(qot=128), INVALID), (dict(hq=-1), INVALID), (dict(rot=256), SHAPE),
])
def test_append_refusals(lib, change, status):
    if status == CUDA and torch.cuda.is_available():
        pytest.skip("would launch")
    a = dict(kv=1, layer=1, K=A, V=B_, dtype=q.F16, T=4, seqs=A, pos=A, table=A, ts=8, ms=4, mp=8, Q=A, hq=8, Qo=B_,
             qot=1024, rot=64)
    a.update(change)
    _, kv = _cache(lib)
    rope = _rope(lib, a["rot"])
    got = lib.qgemm_kv_append(kv if a["kv"] else None, a["layer"], P(a["K"]), 512, 128, P(a["V"]), 512, 128,
                              a["dtype"], a["T"], P(a["seqs"]), P(a["pos"]), P(a["table"]), a["ts"], a["ms"], a["mp"],
                              rope, P(a["Q"]), 1024, 128, a["hq"], P(a["Qo"]), a["qot"], 128, None)
    assert got == status, lib.qgemm_last_error_message()
    lib.qgemm_destroy_kv_cache(kv)
    lib.qgemm_destroy_rope(rope)


@pytest.mark.parametrize("change,status", [
    (dict(), CUDA), (dict(B=0, Q=0), 0), (dict(kv=0), INVALID), (dict(layer=5), INVALID), (dict(dtype=q.BF16), DTYPE),
    (dict(hq=6), INVALID), (dict(hq=0), INVALID), (dict(Q=0), INVALID), (dict(O=0), INVALID), (dict(Q=A + 8), MISALIGNED),
    (dict(qs=1020), MISALIGNED), (dict(os=128), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(window=-1), INVALID), (dict(lens=0), INVALID), (dict(B=5), INVALID), (dict(B=5, seqs=A), CUDA),
    (dict(ms=0), INVALID), (dict(mp=1 << 28), SHAPE), (dict(seqs=A + 2), MISALIGNED), (dict(B=65537, seqs=A), SHAPE),
])
def test_attention_refusals(lib, change, status):
    if status == CUDA and torch.cuda.is_available():
        pytest.skip("would launch")
    a = dict(kv=1, layer=0, Q=A, qs=1024, dtype=q.F16, B=4, hq=8, table=A, ts=8, ms=4, mp=8, lens=A, seqs=0, O=B_, os=1024,
             scale=0.1, window=0)
    a.update(change)
    a["ts"] = max(a["ts"], a["mp"])
    _, kv = _cache(lib)
    got = lib.qgemm_paged_attention(P(a["Q"]), a["qs"], 128, a["dtype"], a["B"], a["hq"], kv if a["kv"] else None,
                                    a["layer"], P(a["table"]), a["ts"], a["ms"], a["mp"], P(a["lens"]), P(a["seqs"]),
                                    P(a["O"]), a["os"], 128, None, a["scale"], a["window"], P(A), 1 << 30, None)
    assert got == status, lib.qgemm_last_error_message()
    lib.qgemm_destroy_kv_cache(kv)


@pytest.mark.parametrize("dtype,pages,page_bytes,scale_bytes,status", [
    (q.F16, 1 << 21, 1 << 16, 0, CUDA),                    # 2^37 bytes in units of a row
    (q.F16, 1 << 21, (1 << 15) + 16, 0, SHAPE),            # 2^36 in units of 16
    (q.F16, (1 << 20) + 1, (1 << 15) + 16, 0, CUDA),       # and half of that
    (q.E4M3, 1 << 21, 1 << 14, (1 << 13) + 4, SHAPE), (q.E4M3, 1 << 21, 1 << 14, 1 << 13, CUDA),
])
def test_attention_counts_offsets_in_units(lib, dtype, pages, page_bytes, scale_bytes, status):
    if status == CUDA and torch.cuda.is_available():
        pytest.skip("would launch")
    row = 128 if dtype == q.E4M3 else 256
    got, kv = _cache(lib, dtype=dtype, layers=1, pages=pages, st=(0, page_bytes, 16 * row, row), ks=A, vs=B_,
                     sst=(0, scale_bytes, 64, 4)) if scale_bytes else \
        _cache(lib, dtype=dtype, layers=1, pages=pages, st=(0, page_bytes, 16 * row, row))
    assert got == 0, lib.qgemm_last_error_message()
    got = lib.qgemm_paged_attention(P(A), 1024, 128, q.F16, 4, 8, kv, 0, P(A), 8, 4, 8, P(A), None, P(B_), 1024, 128,
                                    None, 0.1, 0, P(A), 1 << 30, None)
    assert got == status, lib.qgemm_last_error_message()
    lib.qgemm_destroy_kv_cache(kv)


@pytest.mark.parametrize("change,status", [
    (dict(), CUDA), (dict(n=0, x=0), 0), (dict(kv=0), INVALID), (dict(table=0), INVALID), (dict(ts=4), INVALID),
    (dict(ms=0), INVALID), (dict(mp=0), INVALID), (dict(lens=0), INVALID), (dict(refs=0), INVALID), (dict(x=0), INVALID),
    (dict(x=A + 2), MISALIGNED), (dict(y=A + 1), MISALIGNED), (dict(n=-1), INVALID), (dict(n=1 << 25), SHAPE),
])
def test_page_operation_refusals(lib, change, status):
    if status == CUDA and torch.cuda.is_available():
        pytest.skip("would launch")
    a = dict(kv=1, table=A, ts=8, ms=4, mp=8, lens=A, refs=A, x=A, y=A, n=2)
    a.update(change)
    _, kv = _cache(lib)
    meta = (kv if a["kv"] else None, P(a["table"]), a["ts"], a["ms"], a["mp"], P(a["lens"]), P(a["refs"]))
    for fn in (lib.qgemm_kv_resize, lib.qgemm_kv_fork):
        assert fn(*meta, P(a["x"]), P(a["y"]), a["n"], None) == status, lib.qgemm_last_error_message()
    if not {"x", "y", "n"} & set(change):
        assert lib.qgemm_kv_compact(*meta, None) == status
    if set(change) <= {"x", "y", "n", "kv"}:
        assert lib.qgemm_kv_copy_pages(meta[0], P(a["x"]), P(a["y"]), a["n"], None) == status
    lib.qgemm_destroy_kv_cache(kv)


def test_binding_checks_tensors():
    k = torch.zeros(1, 4, 2, 16, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        q.qgemm_create_kv_cache(k, k.float())
    with pytest.raises(ValueError):
        q.qgemm_create_kv_cache(k.transpose(3, 4), k.transpose(3, 4))
    with pytest.raises(ValueError):
        q.qgemm_create_rope(64, scaling="other")
    x = torch.zeros(4, 2, 128, dtype=torch.float16)
    with pytest.raises(ValueError):                                 # positions of 64 bits
        q.qgemm_rope(x, torch.zeros(4, dtype=torch.int64), q.qgemm_create_rope(64), stream=0)
    with pytest.raises(ValueError):                                 # too few
        q.qgemm_rope(x, torch.zeros(3, dtype=torch.int32), q.qgemm_create_rope(64), stream=0)
    with pytest.raises(ValueError):
        q.qgemm_rope(x.float(), torch.zeros(4, dtype=torch.int32), q.qgemm_create_rope(64), stream=0)


# ------------------------------------------------------------------ the kernels' index arithmetic

SHIM = r"""
#include "kv_index.h"
extern "C" {
int locate(const int32_t *row, int32_t mp, int32_t ps, int32_t pages, int32_t t, int32_t *page, int32_t *off) {
    return kvi::locate(row, mp, ps, pages, t, page, off);
}
int32_t pages_of(int32_t n, int32_t ps) { return kvi::pages_of(n, ps); }
void seen_range(int32_t len, int32_t cap, int32_t window, int32_t *first, int32_t *n) {
    kvi::seen_range(len, cap, window, first, n);
}
int32_t tiles_of(int32_t tokens, int32_t tile) { return kvi::tiles_of(tokens, tile); }
int32_t page_div(int32_t ps, uint32_t t) {
    uint32_t m, s;
    kvi::page_divisor(ps, &m, &s);
    return kvi::page_of(t, m, s);
}
int64_t range_begin(int64_t W, int64_t G, int64_t c) { return kvi::range_begin(W, G, c); }
int64_t range_owner(int64_t W, int64_t G, int64_t x) { return kvi::range_owner(W, G, x); }
}
"""


@pytest.fixture(scope="module")
def idx(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv_index")
    (d / "shim.cpp").write_text(SHIM)
    csrc = os.path.join(os.path.dirname(qbuild.__file__), "csrc")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-I", csrc, str(d / "shim.cpp"), "-o", str(d / "shim.so")], check=True)
    lib = ctypes.CDLL(str(d / "shim.so"))
    lib.range_begin.restype = lib.range_owner.restype = ctypes.c_int64
    lib.range_begin.argtypes = lib.range_owner.argtypes = [ctypes.c_int64] * 3
    return lib


def test_bad_pages_are_not_located(idx):
    row = (ctypes.c_int32 * 4)(3, -1, 8, 7)
    page, off = ctypes.c_int32(), ctypes.c_int32()

    def at(t, pages=8, ps=24):
        return idx.locate(row, 4, ps, pages, t, ctypes.byref(page), ctypes.byref(off))

    assert at(0) and (page.value, off.value) == (3, 0)
    assert at(23) and (page.value, off.value) == (3, 23)
    assert not at(24) and not at(47)                  # -1
    assert not at(48) and not at(71)                  # 8 of 8 pages
    assert at(72) and (page.value, off.value) == (7, 0)
    assert at(95) and (page.value, off.value) == (7, 23)
    for t in (96, 97, 2 ** 31 - 1, -1, -2 ** 31):     # outside the row: the row is not read there
        assert not at(t)


def test_counts_at_the_ends(idx):
    for ps in (1, 2, 16, 24, 65536):
        for n in (0, 1, ps - 1, ps, ps + 1, 2 ** 31 - 1):
            assert idx.pages_of(n, ps) == -(-n // ps)
            assert idx.tiles_of(n, ps) == max(1, -(-n // ps))
    first, n = ctypes.c_int32(), ctypes.c_int32()
    for length, cap, window, want in ((10, 64, 0, (0, 10)), (10, 64, 4, (6, 10)), (10, 64, 10, (0, 10)), (0, 64, 3, (0, 0)),
                                      (-5, 64, 0, (0, 0)), (100, 64, 0, (0, 64)), (100, 64, 8, (56, 64)),
                                      (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, (0, 2 ** 31 - 1))):
        idx.seen_range(length, cap, window, ctypes.byref(first), ctypes.byref(n))
        assert (first.value, n.value) == want


def test_page_division(idx):
    rng = random.Random(1)
    for ps in list(range(1, 300)) + [2 ** k + e for k in range(8, 17) for e in (-1, 0, 1) if 2 ** k + e <= 65536]:
        ts = {0, 1, ps - 1, ps, ps + 1, 2 ** 31 - 1, 2 ** 31 - 2, (2 ** 31 - 1) // ps * ps, max(0, (2 ** 31 - 1) // ps * ps - 1)}
        for t in ts | {rng.randrange(2 ** 31) for _ in range(40)}:
            assert idx.page_div(ps, t) == t // ps


def test_ranges_cover_every_tile_once(idx):
    rng = random.Random(3)
    for _ in range(300):
        sizes = [rng.choice([1, 1, 2, rng.randint(1, 40), rng.randint(1, 3000)]) for _ in range(rng.randint(1, 30))]
        W = sum(sizes)
        G = min(rng.choice([1, 2, 7, 152]), W)
        begin = [idx.range_begin(W, G, c) for c in range(G + 1)]
        assert begin[0] == 0 and begin[G] == W
        assert all(0 <= b - a - W // G <= 1 for a, b in zip(begin, begin[1:]))
        for x in rng.sample(range(W), min(W, 50)) + begin[:-1] + [b - 1 for b in begin[1:]]:
            c = idx.range_owner(W, G, x)
            assert begin[c] <= x < begin[c + 1]
        # the pieces of a unit are those of consecutive CTAs, and a CTA has at most two cut ones:
        # one that began before its range and one that goes on after it
        at, slots = 0, set()
        for n in sizes:
            a, b = idx.range_owner(W, G, at), idx.range_owner(W, G, at + n - 1)
            if a != b:
                for c in range(a, b + 1):
                    assert begin[c] < at + n and begin[c + 1] > at
                    slot = 2 * c + (c == a)
                    assert slot not in slots and slot < 2 * G
                    slots.add(slot)
            at += n
    big = 65536 * 65536 * 4
    assert idx.range_owner(big, 152, big - 1) == 151 and idx.range_begin(big, 152, 152) == big


# ----------------------------------------------------------------------- the tests' own references

def test_reference_rotation_is_orthogonal_and_inverts():
    x = torch.randn(5, 3, 96, dtype=torch.float64)
    pos = torch.tensor([0, 1, 7, 100000, 2 ** 31 - 1])
    for inter in (False, True):
        y, _ = ref.rotate(x, pos, 48, inter)
        assert torch.equal(y[0], x[0]) and torch.equal(y[..., 48:], x[..., 48:])
        z, _ = ref.rotate(y, pos, 48, inter, inverse=True)
        assert (z - x).abs().max() < 1e-12


def test_reference_inverse_is_the_gradient():
    """Against differences of the loss <g, rotate(x)>."""
    g, x = torch.randn(2, 1, 16, dtype=torch.float64), torch.randn(2, 1, 16, dtype=torch.float64)
    pos = torch.tensor([3, 12345])
    grad, _ = ref.rotate(g, pos, 12, True, inverse=True, mscale=1.3)
    for i in range(16):
        h = torch.zeros_like(x)
        h[..., i] = 1e-6
        up, _ = ref.rotate(x + h, pos, 12, True, mscale=1.3)
        dn, _ = ref.rotate(x - h, pos, 12, True, mscale=1.3)
        diff = ((up - dn) * g).sum(-1).sum(-1) / 2e-6
        want = grad[..., i][:, 0] if i < 12 else g[..., i][:, 0]
        assert (diff - want).abs().max() < 1e-7


def test_reference_pages_keep_their_counts():
    rng = random.Random(5)
    p = ref.Pages([[-1] * 12 for _ in range(10)], [0] * 10, [0] * 40, 8)
    for _ in range(300):
        op = rng.random()
        if op < 0.6:
            seqs = rng.sample(range(10), rng.randint(1, 5))
            p.resize(seqs, [rng.choice([0, p.lens[s] + 1, rng.randint(0, 96)]) if p.lens[s] < 96 else 0 for s in seqs])
        elif op < 0.85:
            two = rng.sample(range(10), 4)
            p.fork([two[0], two[0], two[1]][:2], two[2:])
        else:
            p.compact()
        held = [0] * 40
        for s in range(10):
            n = p.of(p.lens[s])
            assert all(0 <= x < 40 for x in p.table[s][:n]) and all(x == -1 for x in p.table[s][n:])
            for x in p.table[s][:n]:
                held[x] += 1
        assert held == p.refs


def test_every_tile_has_one_cta(idx):
    """The attention's walk over its range, restated: with a unit counting `extra` tiles beyond its own, every tile
    is computed by one CTA, and the parts of a cut unit are those of consecutive CTAs."""
    rng = random.Random(7)
    for _ in range(200):
        extra = rng.choice([0, 1, 2, 3])
        units = [rng.choice([1, 1, 2, rng.randint(1, 40), rng.randint(1, 500)]) for _ in range(rng.randint(1, 40))]
        starts, at = [], 0
        for n in units:
            starts.append(at)
            at += n + extra
        W = at
        G = min(rng.choice([1, 2, 7, 152, 304]), W)
        seen = [[] for _ in units]
        for c in range(G):
            begin, end = idx.range_begin(W, G, c), idx.range_begin(W, G, c + 1)
            u = max(i for i, s in enumerate(starts) if s <= begin)
            tile = max(0, begin - starts[u] - extra)
            pos = starts[u] + extra + tile
            while pos < end:
                seen[u].append((tile, c))
                pos, tile = pos + 1, tile + 1
                if tile == units[u]:
                    u, tile, pos = u + 1, 0, pos + extra
        for u, n in enumerate(units):
            assert [t for t, _ in seen[u]] == list(range(n))
            t0 = starts[u] + extra
            first, last = idx.range_owner(W, G, t0), idx.range_owner(W, G, t0 + n - 1)
            assert sorted({c for _, c in seen[u]}) == list(range(first, last + 1))
            for c in range(first, last + 1):          # who opens the unit, as each CTA sees it
                assert (t0 >= idx.range_begin(W, G, c)) == (c == first)


def test_parts_are_merged_once_each():
    """The merging of a cut unit's n parts, restated: whatever order they arrive in, one part's owner finishes with
    all of them merged in order, every counter is back at zero, and no part is read after it was replaced."""
    rng = random.Random(11)
    fan, levels = 32, 2
    for n in [2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 152, 304, 1023, 1024]:
        for _ in range(3):
            order = list(range(n))
            rng.shuffle(order)
            held, counters, finished = {}, {}, []
            for first in order:
                i, stride, value = first, 1, [first]
                for level in range(levels):
                    held[i] = value
                    i0 = i - i % (fan * stride)
                    members = min(fan, (n - i0 + stride - 1) // stride)
                    counters[level, i0] = counters.get((level, i0), 0) + 1
                    if counters[level, i0] != members:
                        break
                    counters[level, i0] = 0
                    value = sum((held.pop(i0 + k * stride) for k in range(members)), [])
                    if i0 == 0 and members * stride >= n:
                        finished.append(value)
                        break
                    i, stride = i0, stride * fan
                else:
                    raise AssertionError("more levels needed")
            assert finished == [list(range(n))] and not any(counters.values())

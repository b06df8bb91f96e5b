"""Rotary positions and the paged cache's append on the GPU against 64-bit references.

16-bit results: ref.rope_tolerance.  E4M3: each stored value is within half an E4M3 step (2^-4 of the value,
2^-10 of its block's unit below E4M3's normal range) of the fp32 rotation, which is off by the same
arithmetic error; where the amax lies at a power of two the scale may fall on either side, so codes are
judged by the values they stand for and the scale by its definition with that slack.
"""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu

SCALINGS = {"none": {}, "linear": dict(scaling="linear", factor=4.0),
            "by_parts": dict(scaling="by_parts", factor=8.0, original_len=4096)}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from block_scaled_quantized_tcgen05_gb300 import build
    build.build()
    q.load_library()
    return torch.device("cuda:0")


def _clean(what=""):
    assert q.qgemm_poll_device_error() == 0, what


def _close(got, want, mag, what):
    tol = ref.rope_tolerance(want, mag, got.dtype)
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: {(err / tol).max().item():.3f} of the tolerance"


def _positions(T, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, 2 ** 20, (T,), generator=g, dtype=torch.int32)
    ends = torch.tensor([0, 2 ** 31 - 1, -3, 1, 131071], dtype=torch.int32)
    p[:min(T, 5)] = ends[:min(T, 5)]
    return p


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,H,d,rot,inter,scaling,inverse", [
    (1, 1, 128, 128, False, "none", False), (5, 40, 128, 128, False, "by_parts", False),
    (333, 3, 64, 32, True, "linear", True), (17, 7, 96, 48, False, "linear", True),
    (17, 7, 96, 38, False, "none", False), (9, 5, 80, 40, False, "none", True), (9, 5, 80, 34, True, "none", False),
    (1000, 12, 256, 256, False, "by_parts", False), (4, 2, 256, 102, True, "none", True),
    (33, 5, 72, 32, False, "none", False), (33, 5, 104, 96, False, "linear", True), (65, 9, 112, 64, True, "none", False),
    (3, 2, 2, 2, False, "none", False), (3, 3, 50, 50, False, "linear", False), (700, 48, 128, 64, True, "none", False),
])
def test_rope_matches(dev, dtype, T, H, d, rot, inter, scaling, inverse):
    g = torch.Generator().manual_seed(T + d + rot)
    x = torch.randn(T, H, d, generator=g).to(dtype)
    pos = _positions(T, T)
    m = 1.25 if scaling == "by_parts" else 1.0
    rope = q.qgemm_create_rope(rot, interleaved=inter, mscale=m, **SCALINGS[scaling])
    want, mag = ref.rotate(x, pos, rot, inter, inverse, m, **{**SCALINGS[scaling]})
    xd = x.to(dev)
    y = torch.full_like(xd, float("nan"))
    assert q.qgemm_rope(xd, pos.to(dev), rope, out=y, inverse=inverse) is y
    _clean()
    _close(y, want, mag, "out of place")
    again = xd.clone()
    q.qgemm_rope(again, pos.to(dev), rope, inverse=inverse)           # in place
    assert torch.equal(again, y)
    _clean()


@pytest.mark.parametrize("rot,inter", [(128, False), (100, False), (128, True)])
def test_rope_strides_alignment_and_guards(dev, rot, inter):
    """Heads outside tokens, padded rows, a base two bytes off: only the rows themselves are written."""
    T, H, d = 37, 6, 128
    rope = q.qgemm_create_rope(rot, interleaved=inter)
    pos = torch.arange(T, dtype=torch.int32) * 1000
    for shift, pad, swap in ((0, 0, True), (1, 3, False), (8, 8, True)):
        buf = torch.randn(T * H * (d + pad) + 16, dtype=torch.float16, device=dev)
        out = torch.full_like(buf, 7.0)
        shape, st = ((T, H, d), (d + pad, T * (d + pad), 1)) if swap else ((T, H, d), (H * (d + pad), d + pad, 1))
        x = buf.as_strided(shape, st, shift)
        y = out.as_strided(shape, st, shift)
        q.qgemm_rope(x, pos.to(dev), rope, out=y)
        want, mag = ref.rotate(x.cpu(), pos, rot, inter)
        _close(y, want, mag, f"shift {shift}")
        y.fill_(7.0)
        assert bool((out == 7.0).all())
    _clean()


def test_rope_strides_past_31_bits(dev):
    """Heads more than 2^31 bytes apart, of the input and of the output."""
    T, H, d, far = 5, 2, 128, 2 ** 30 + 64
    x = torch.empty(far + T * d, dtype=torch.float16, device=dev).as_strided((T, H, d), (d, far, 1))
    y = torch.empty(far + T * d, dtype=torch.float16, device=dev).as_strided((T, H, d), (d, far, 1))
    x.copy_(torch.randn(T, H, d))
    pos = torch.arange(T, dtype=torch.int32) * 777
    q.qgemm_rope(x, pos.to(dev), q.qgemm_create_rope(d), out=y)
    _clean()
    _close(y, *ref.rotate(x.cpu(), pos, d), "far heads")


def test_rope_gradient_against_differences(dev):
    """The inverse on the GPU against differences of <g, rotate(x)> computed by the forward in steps an
    fp16 value represents exactly (the map is linear, so the step's size does not matter)."""
    T, H, d, rot = 3, 2, 32, 24
    rope = q.qgemm_create_rope(rot, mscale=1.5)
    pos = torch.tensor([2, 77, 40000], dtype=torch.int32, device=dev)
    g = torch.randn(T, H, d, device=dev).to(torch.float16)
    grad = q.qgemm_rope(g, pos, rope, out=torch.empty_like(g), inverse=True)
    for i in range(d):
        e = torch.zeros(T, H, d, dtype=torch.float16, device=dev)
        e[..., i] = 1.0
        up = q.qgemm_rope(e, pos, rope, out=torch.empty_like(e)).double()
        dn = q.qgemm_rope(-e, pos, rope, out=torch.empty_like(e)).double()
        diff = ((up - dn) / 2 * g.double()).sum(-1)
        # the forward's column has two entries up to 1.5, each rounded by 2^-11 (and 2^-21), times g
        tol = 2 * 1.5 * 2.0 ** -10 * g.double().abs().amax(-1) + 2.0 ** -11 * grad[..., i].double().abs()
        assert bool(((diff - grad[..., i].double()).abs() <= tol).all())
    _clean()


@pytest.mark.parametrize("T,H,d,rot,inter", [
    (5003, 1, 256, 254, False), (2500, 13, 64, 24, False), (1201, 40, 128, 50, False), (2011, 7, 80, 38, False),
    (907, 6, 120, 96, False), (1203, 40, 96, 38, True), (3001, 5, 128, 126, True), (2003, 3, 90, 90, False),
])
def test_rope_parts_over_many_rounds(dev, T, H, d, rot, inter):
    """Blocks of several tokens and rounds, in place; infinities past the rotated part stay there."""
    g = torch.Generator().manual_seed(d + rot)
    x = torch.randn(T, H, d, generator=g).half()
    if rot < d:
        x[::3, :, rot] = float("inf")
        x[1::3, :, d - 1] = -float("inf")
    pos = _positions(T, d)
    rope = q.qgemm_create_rope(rot, interleaved=inter)
    y = x.to(dev)
    q.qgemm_rope(y, pos.to(dev), rope, out=y)
    want, mag = ref.rotate(x, pos, rot, inter)
    assert torch.equal(y.cpu()[..., rot:], x[..., rot:])
    _close(y[..., :rot], want[..., :rot], mag[..., :rot], "rotated part")
    _clean()


def test_rope_nothing_to_do(dev):
    rope = q.qgemm_create_rope(64)
    x = torch.empty(0, 4, 64, dtype=torch.float16, device=dev)
    q.qgemm_rope(x, torch.empty(0, dtype=torch.int32, device=dev), rope)
    _clean()


# ------------------------------------------------------------------------------------- append

def make_cache(dev, dtype, e4m3, layers, pages, heads, page, d, order="lphtd"):
    """Planes full of a marker, in the order of dimensions given, and their view."""
    shape = dict(l=layers, p=pages, h=heads, t=page)
    perm = [c for c in order if c != "d"]
    back = [perm.index(c) for c in "lpht"]

    def plane(inner, dt, fill):
        return torch.full([shape[c] for c in perm] + [inner], fill, dtype=dt, device=dev).permute(*back, 4)

    if e4m3:
        k, v = (plane(d, torch.uint8, 0x11) for _ in "kv")
        ks, vs = (plane(4, torch.uint8, 0x22) for _ in "kv")
        return dict(k=k, v=v, ks=ks, vs=vs, kv=q.qgemm_create_kv_cache(k, v, ks, vs))
    k, v = (plane(d, dtype, 3.0) for _ in "kv")
    return dict(k=k, v=v, kv=q.qgemm_create_kv_cache(k, v))


def _check_e4m3(codes, scales, x, mag, dtype, what):
    """codes [T, H, d] and scale bytes [T, H, >= d / 32] against the exact rows x."""
    d = x.shape[-1]
    slack = (2.0 ** -21 * mag).unflatten(-1, (-1, 32)).amax(-1)
    amax = x.abs().unflatten(-1, (-1, 32)).amax(-1)
    byte = scales[..., :d // 32].cpu().to(torch.int64)
    least = 127 - (15 if dtype == torch.float16 else 127)

    def scale_of(a):
        e = torch.where(a > 0, torch.frexp(a.clamp(min=1e-300))[1] - 1 - 8 + 127, 127)
        return torch.where(a > 0, e.clamp(min=least), e)

    lo, hi = scale_of((amax - slack).clamp(min=0)), scale_of(amax + slack)
    near_zero = amax <= slack
    assert bool(((byte >= lo) & (byte <= hi) | near_zero).all()), f"{what}: scales"
    unit = torch.exp2(byte.double() - 127).repeat_interleave(32, -1)
    v = ref.e4m3(codes) * unit
    xc = x.clamp(min=-448 * unit, max=448 * unit)
    tol = torch.maximum(2.0 ** -4 * xc.abs(), 2.0 ** -10 * unit) * (1 + 2.0 ** -10) + 2 * 2.0 ** -21 * mag
    err = (v - xc).abs()
    assert bool((err <= tol).all()), f"{what}: {(err / tol).max().item():.3f} of the tolerance"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,hq,hkv,page,rot,inter,order", [
    (128, 8, 2, 16, 128, False, "lphtd"), (128, 7, 1, 24, 64, True, "plhtd"), (64, 12, 4, 5, 64, False, "lpthd"),
    (64, 0, 3, 1, 0, False, "lphtd"), (128, 32, 8, 64, 40, False, "lpthd"),
    (128, 4, 2, 16, 96, False, "lphtd"), (128, 3, 1, 32, 32, False, "plhtd"), (64, 5, 5, 16, 32, True, "lphtd"),
    (64, 2, 1, 8, 16, False, "lphtd"), (128, 6, 3, 16, 100, True, "lphtd"),
])
def test_append_matches(dev, dtype, e4m3, d, hq, hkv, page, rot, inter, order):
    layers, lens, new = 3, [0, 5, 2 * page + 1, 3], [4, 1, 2 * page + 3, 0]
    total = [a + b for a, b in zip(lens, new)]
    mp = max(-(-n // page) for n in total) + 1
    used = sum(-(-n // page) for n in total)
    c = make_cache(dev, dtype, e4m3, layers, used + 2, hkv, page, d, order)
    g = torch.Generator().manual_seed(d + page)
    ids = torch.randperm(used + 2, generator=g).to(torch.int32)
    table = torch.full((6, mp), -1, dtype=torch.int32)
    rows, at = [4, 0, 3, 1], 0
    for s, n in zip(rows, total):
        k = -(-n // page)
        table[s, :k] = ids[at:at + k]
        at += k
    seqs = torch.cat([torch.full((b,), s, dtype=torch.int32) for s, b in zip(rows, new)])
    pos = torch.cat([torch.arange(a, a + b, dtype=torch.int32) for a, b in zip(lens, new)])
    T = len(seqs)
    x = torch.randn(T, hq + 2 * hkv, d, generator=g)
    x[:, :, 32:64] *= 2.0 ** torch.randint(-12, 6, (T, hq + 2 * hkv, 1), generator=g).float()
    x = x.to(dtype)
    x[0, -1, :32] = 0.0                                                # an all-zero block
    xq, xk, xv = x.to(dev).split([hq, hkv, hkv], 1)
    rope = q.qgemm_create_rope(rot, interleaved=inter) if rot else None
    before = {n: c[n].clone() for n in c if n != "kv"}
    out = torch.empty(T, hq, d, dtype=dtype, device=dev)
    q.qgemm_kv_append(c["kv"], 1, xk, xv, seqs.to(dev), pos.to(dev), table.to(dev), rope=rope,
                      **(dict(Q=xq, Q_out=out) if hq else {}))
    _clean()
    turn = (lambda t: ref.rotate(t, pos, rot, inter)) if rot else (lambda t: (t.double(), t.double().abs()))
    if hq:
        _close(out, *turn(x[:, :hq]), "queries")
    kx, kmag = turn(x[:, hq:hq + hkv])
    vx = x[:, hq + hkv:].double()
    pg = table[seqs.long(), (pos // page).long()].long().to(dev)
    off = (pos % page).long().to(dev)
    if e4m3:
        _check_e4m3(c["k"][1, pg, :, off], c["ks"][1, pg, :, off], kx, kmag, dtype, "keys")
        _check_e4m3(c["v"][1, pg, :, off], c["vs"][1, pg, :, off], vx, torch.zeros_like(vx), dtype, "values")
        if T:
            assert int(c["vs"][1, pg[0], -1, off[0], 0]) == 127
    else:
        _close(c["k"][1, pg, :, off], kx, kmag, "keys")
        assert torch.equal(c["v"][1, pg, :, off].cpu(), x[:, hq + hkv:])
    # nothing else is written
    for n, t in before.items():
        now = c[n].clone()
        live = d // 32 if n in ("ks", "vs") else d
        now[1, pg, :, off, :live] = t[1, pg, :, off, :live]
        assert torch.equal(now.view(torch.uint8) if now.is_contiguous() else now, t.view(torch.uint8) if t.is_contiguous() else t), n


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,hq,hkv,rot,inter,T", [
    (128, 5, 2, 100, False, 1500), (64, 3, 1, 24, False, 2000), (128, 8, 2, 102, True, 1100), (128, 3, 3, 96, False, 1300),
])
def test_append_parts_over_many_rounds(dev, e4m3, d, hq, hkv, rot, inter, T):
    """One long sequence, more tokens than one round of a block, rotated in part."""
    page = 24
    pages = -(-T // page)
    c = make_cache(dev, torch.float16, e4m3, 1, pages, hkv, page, d)
    g = torch.Generator().manual_seed(rot)
    x, k, v = (torch.randn(T, h, d, generator=g).half() for h in (hq, hkv, hkv))
    table = torch.randperm(pages, generator=g).to(torch.int32)[None]
    pos = torch.arange(T, dtype=torch.int32)
    rope = q.qgemm_create_rope(rot, interleaved=inter)
    out = torch.empty(T, hq, d, dtype=torch.float16, device=dev)
    q.qgemm_kv_append(c["kv"], 0, k.to(dev), v.to(dev), torch.zeros(T, dtype=torch.int32, device=dev), pos.to(dev),
                      table.to(dev), rope=rope, Q=x.to(dev), Q_out=out)
    _clean()
    _close(out, *ref.rotate(x, pos, rot, inter), "queries")
    want, mag = ref.rotate(k, pos, rot, inter)
    pg, off = table[0, (pos // page).long()].long().to(dev), (pos % page).long().to(dev)
    if e4m3:
        _check_e4m3(c["k"][0, pg, :, off], c["ks"][0, pg, :, off], want, mag, torch.float16, "keys")
        _check_e4m3(c["v"][0, pg, :, off], c["vs"][0, pg, :, off], v.double(), torch.zeros_like(want), torch.float16,
                    "values")
    else:
        _close(c["k"][0, pg, :, off], want, mag, "keys")
        assert torch.equal(c["v"][0, pg, :, off].cpu(), v)


def test_append_special_values(dev):
    """NaN becomes E4M3's NaN in its place alone; an infinity, its block's largest, stays infinite."""
    for dtype in (torch.float16, torch.bfloat16):
        c = make_cache(dev, dtype, True, 1, 1, 1, 4, 64)
        x = torch.randn(1, 1, 64).to(dtype)
        x[0, 0, 3], x[0, 0, 40] = float("nan"), float("-inf")
        zero = torch.zeros(1, dtype=torch.int32, device=dev)
        q.qgemm_kv_append(c["kv"], 0, x.to(dev), x.to(dev), zero, zero, zero.view(1, 1))
        _clean()
        v = ref.dequant(c["v"][0, 0, 0, 0], c["vs"][0, 0, 0, 0], dtype)
        assert bool(v[3].isnan()) and int(v.isnan().sum()) == 1 and v[40] == float("-inf")
        assert bool(((v[:32] - x[0, 0, :32].double()).abs()[x[0, 0, :32].isfinite()] <= 0.25).all())


def test_append_skips_bad_indices(dev):
    """Sequences, positions and pages out of range: their tokens are skipped, the others stored, and the error
    word says so."""
    c = make_cache(dev, torch.float16, False, 1, 4, 2, 8, 64)
    before = c["k"].clone()
    table = torch.tensor([[0, -1], [9, 3], [2, 1]], dtype=torch.int32, device=dev)
    seqs = torch.tensor([0, 0, 1, 1, 2, 3, -1, 2, 2], dtype=torch.int32, device=dev)
    pos = torch.tensor([1, 8, 0, 9, 16, 0, 0, -1, 15], dtype=torch.int32, device=dev)
    x = torch.randn(9, 2, 64, device=dev).to(torch.float16)
    q.qgemm_kv_append(c["kv"], 0, x, x, seqs, pos, table)
    assert q.qgemm_poll_device_error() == 64
    want = before.clone()
    for t, (p, r) in {0: (0, 1), 3: (3, 1), 8: (1, 7)}.items():
        want[0, p, :, r] = x[t]
    assert torch.equal(c["k"], want)

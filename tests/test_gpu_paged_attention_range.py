"""Single-token attention with bf16 values over the type's whole range: large values of vanishing weight, and values
near its end.

Tolerances, beside the output's own rounding (HALF) and that of the scores (kv_reference.attend_tolerance's): a weight
is held to 2^-15 of itself and 2^-125 of the largest one, which in bf16 is far below what any value makes visible;
the steps of an E4M3 cache whose scales are halves hold it to 2^-38 of the largest, and have values up to 448.
"""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests import kv_reference as ref
from tests.test_gpu_paged_attention import Problem, _clean, dev  # noqa: F401

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
HEADS = [(128, 1, 1), (64, 4, 1), (128, 8, 1), (64, 16, 1), (128, 3, 1), (64, 8, 2), (128, 40, 2)]


def tolerance(o, D, S, n, v, e4m3):
    top = v.abs().amax(0)                                            # of each element
    least = 2.0 ** -125 * top + (2.0 ** -38 * top.clamp(max=448.0) if e4m3 else 0.0)
    score = (16 * 2.0 ** -22 + 2.0 ** -22) * max(S, 1.0)
    return ref.HALF[BF16] * (1 + 2.0 ** -8) * o.abs() + (2.0 ** -15 + 2 * score) * D + n * least + ref.TINY[BF16]


def check(p, o, l):
    g = p.hq // p.hkv
    for b, n in enumerate(p.lens):
        for h in range(p.hkv):
            k, v = (x[:, h] for x in p.seen[b])
            want, lse, D, S = ref.attend(p.q[b, h * g:(h + 1) * g], k, v, p.d ** -0.5)
            assert bool((want.abs() < 2.0 ** 127).all())
            got = o[b, h * g:(h + 1) * g].cpu().double()
            tol = tolerance(want, D, S, n, v, p.e4m3)
            assert bool(got.isfinite().all()), f"b {b} n {n} h {h}: {got[~got.isfinite()][:4]}"
            err = (got - want).abs()
            assert bool((err <= tol).all()), f"b {b} n {n} h {h}: {(err / tol).max().item():.3g} of the tolerance"
            assert bool(((l[b, h * g:(h + 1) * g].cpu().double() - lse).abs() <= ref.lse_tolerance(lse, S)).all())


def place(p, b, t):
    return p.table[p.rows[b], t // p.page].long(), t % p.page


def set_codes(p, b, t, name, codes=None, scales=None):
    """Rows t (a tensor of token numbers) of sequence b of an E4M3 cache: codes, scale bytes or both, and what they stand for."""
    pg, off = place(p, b, t)
    if codes is not None:
        getattr(p, name)[1, pg, :, off] = codes
    if scales is not None:
        getattr(p, name + "s")[1, pg, :, off] = scales
    x = ref.dequant(getattr(p, name)[1, pg, :, off], getattr(p, name + "s")[1, pg, :, off], p.dtype)
    p.seen[b]["kv".index(name)][t] = x


def set_rows(p, b, t, name, x):
    pg, off = place(p, b, t)
    getattr(p, name)[1, pg, :, off] = x
    p.seen[b]["kv".index(name)][t] = x.double()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,hq,hkv", HEADS)
@pytest.mark.parametrize("at,batch", [(5, 1), (130, 1), (130, 400)])
def test_a_large_value_of_vanishing_weight(dev, e4m3, d, hq, hkv, at, batch):  # noqa: F811
    """Token 0 outweighs the others by about e^45 and its own values are zero; token `at` has values whose share of the sum,
    e^-45 of them, is far below 2^-38 of them: in the same step; in another part of the sequence; and in a later step of
    the same part (a batch whose sequences are not cut)."""
    p = Problem(dev, [300] * batch, hq, hkv, d, 16, BF16, e4m3, seed=at + hq)
    base = p.q[0, 0].float()
    p.q[0] = (base * (1 + torch.arange(hq)[:, None] / 64)).to(BF16)
    first, it = torch.tensor([0]), torch.tensor([at])
    key = (base * (45 * d ** 0.5 / float(base.square().sum()))).expand(1, hkv, d)
    if e4m3:
        set_codes(p, 0, first, "k", key.to(torch.float8_e4m3fn).view(torch.uint8), torch.full((1, hkv, 4), 127, dtype=torch.uint8))
        set_codes(p, 0, first, "v", torch.zeros(1, hkv, d, dtype=torch.uint8))
        b = torch.full((1, hkv, 4), 120, dtype=torch.uint8)
        b[..., 1] = 187
        set_codes(p, 0, it, "v", None, b)
    else:
        set_rows(p, 0, first, "k", key.to(BF16))
        set_rows(p, 0, first, "v", torch.zeros(1, hkv, d, dtype=BF16))
        v = p.seen[0][1][it].to(BF16)
        v[..., 7], v[..., 9], v[..., 40] = 1e12, -1e9, 1e30
        set_rows(p, 0, it, "v", v)
    o, l = p.run()
    _clean()
    check(p, o, l)


@pytest.mark.parametrize("d,hq,hkv", HEADS)
def test_values_near_the_end_of_the_range(dev, d, hq, hkv):  # noqa: F811
    """One token of 1e35 gives 1e35, and the mean of hundreds of them is one."""
    p = Problem(dev, [1, 300, 40, 700], hq, hkv, d, 16, BF16, False, seed=31)
    g = torch.Generator().manual_seed(d)
    for b, n in enumerate(p.lens):
        v = (1e35 * (0.5 + torch.rand(n, hkv, d, generator=g)) * (torch.randint(0, 2, (n, hkv, 1), generator=g) * 2 - 1)).to(BF16)
        set_rows(p, b, torch.arange(n), "v", v)
    o, l = p.run()
    _clean()
    check(p, o, l)


@pytest.mark.parametrize("d,hq,hkv", HEADS)
def test_value_scales_near_the_end_of_the_range(dev, d, hq, hkv):  # noqa: F811
    """E4M3 values of up to 5e36 in one block of a few tokens, among others of ordinary size: every element is right, those
    of the other blocks too, with the large tokens before, between and after the others and in part of a cut sequence."""
    p = Problem(dev, [1, 300, 20, 6000, 129], hq, hkv, d, 16, BF16, True, seed=32)
    g = torch.Generator().manual_seed(d + 1)
    for b, big in enumerate([[0], [3, 20, 131, 132, 260], [19], [0, 1500, 1501, 5999], [128]]):
        t = torch.tensor(big)
        codes = p.v[1, place(p, b, t)[0], :, place(p, b, t)[1]].clone()
        codes[(codes & 0x78) == 0x78] = 0x30                         # below 256
        s = torch.full((len(big), hkv, 4), 120, dtype=torch.uint8)
        s[..., 1] = torch.randint(225, 242, (len(big), hkv), generator=g, dtype=torch.uint8)
        set_codes(p, b, t, "v", codes, s)
    o, l = p.run()
    _clean()
    check(p, o, l)

"""An infinite value of a weight below what fp32 holds, e^-200 of the largest, is an infinite sum wherever the two tokens lie: in
one step, in steps of one warp (either first), in different warps, in parts of the sequence that different blocks take."""
import pytest
import torch

from tests.test_gpu_paged_attention import Problem, _clean, dev  # noqa: F401

pytestmark = pytest.mark.gpu

PLACES = [(5, 0, 300, 1), (50, 0, 300, 1), (130, 0, 300, 400), (0, 130, 300, 400), (290, 0, 300, 1), (0, 290, 300, 1),
          (39000, 5, 40000, 1), (5, 39000, 40000, 1)]


@pytest.mark.parametrize("e4m3,dtype", [(False, torch.float16), (False, torch.bfloat16), (True, torch.float16), (True, torch.bfloat16)])
@pytest.mark.parametrize("d,hq", [(128, 1), (64, 7), (128, 12)])
@pytest.mark.parametrize("at,top,n,batch", PLACES)
def test_infinite_values_of_vanishing_weight(dev, e4m3, dtype, d, hq, at, top, n, batch):  # noqa: F811
    p = Problem(dev, [n] * batch, hq, 1, d, 16, dtype, e4m3, seed=at + hq)
    base = p.q[0, 0].float()
    p.q[0] = (base * (1 + torch.arange(hq)[:, None] / 64)).to(dtype)
    key = base * (200 * d ** 0.5 / float(base.square().sum()))
    (pt, ot), (pa, oa) = ((int(p.table[0, t // 16]), t % 16) for t in (top, at))
    if e4m3:
        p.k[1, pt, 0, ot], p.ks[1, pt, 0, ot] = (key / 4).to(torch.float8_e4m3fn).view(torch.uint8), 129
        p.vs[1, pt, 0, ot, 0] = 120
        p.v[1, pa, 0, oa, 7], p.v[1, pa, 0, oa, 9] = 0x7E, 0xFE      # +-448 times 2^127
        for e in (*range(7), 8, *range(10, 32)):
            p.v[1, pa, 0, oa, e] = 0
        p.vs[1, pa, 0, oa, 0] = 254
    else:
        p.k[1, pt, 0, ot] = key.to(dtype)
        p.v[1, pa, 0, oa, 7], p.v[1, pa, 0, oa, 9] = float("inf"), float("-inf")
    o, l = p.run()
    _clean()
    o = o.cpu().float()
    assert bool((o[0, :, 7] == float("inf")).all()) and bool((o[0, :, 9] == float("-inf")).all())
    assert int((~o[0].isfinite()).sum()) == 2 * hq and bool(l.isfinite().all())
    assert batch == 1 or bool(o[1:].isfinite().all())

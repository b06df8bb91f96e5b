"""One token, or one head, whose stride in that dimension is odd (it is never stepped): the calls take it, and on the
GPU give the bits of a dense tensor."""
import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests.test_gpu_paged_attention import Problem, _clean, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def odd(x, dim):
    """x with a stride of 3 in its dimension `dim` of one."""
    st = list(x.stride())
    st[dim] = 3
    return x.as_strided(x.shape, st)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,hq,hkv,dim", [(1, 8, 2, 0), (3, 1, 1, 1), (1, 1, 1, 0)])
def test_attention(dev, e4m3, B, hq, hkv, dim):  # noqa: F811
    p = Problem(dev, [200, 3, 77][:B], hq, hkv, 128, 16, torch.float16, e4m3, seed=41)
    kv = p.upload()
    want, _ = p.run(kv=kv)
    qd = p.q.to(dev)
    o = torch.empty_like(qd)
    q.qgemm_paged_attention(odd(qd, dim), kv, 1, p.table.to(dev), p.seq_lens.to(dev), odd(o, dim))
    _clean()
    assert torch.equal(o, want)


@pytest.mark.parametrize("T,H,dim", [(1, 8, 0), (50, 1, 1), (1, 1, 1)])
def test_rope_and_append(dev, T, H, dim):  # noqa: F811
    rope = q.qgemm_create_rope(128)
    x, k, v = (torch.randn(T, H, 128, device=dev).half() for _ in "xkv")
    pos, seqs = torch.arange(T, dtype=torch.int32, device=dev), torch.zeros(T, dtype=torch.int32, device=dev)
    want = q.qgemm_rope(x, pos, rope, out=torch.empty_like(x))
    y = torch.empty_like(x)
    q.qgemm_rope(odd(x, dim), pos, rope, out=odd(y, dim))
    assert torch.equal(y, want)
    table = torch.arange(4, dtype=torch.int32, device=dev)[None]
    planes = []
    for f in (lambda t: t, lambda t: odd(t, dim)):
        kp, vp = (torch.zeros(1, 4, H, 16, 128, dtype=torch.float16, device=dev) for _ in "kv")
        y = torch.empty_like(x)
        q.qgemm_kv_append(q.qgemm_create_kv_cache(kp, vp), 0, f(k), f(v), seqs, pos, table, rope=rope, Q=f(x), Q_out=f(y))
        planes.append((kp, vp, y))
    _clean()
    assert all(torch.equal(a, b) for a, b in zip(*planes)) and torch.equal(planes[0][2], want)

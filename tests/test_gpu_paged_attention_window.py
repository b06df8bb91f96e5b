"""Sliding windows over pages of a multiple of 16 tokens (where a step of the kernel lies in one page): windows that begin
inside a step, at its ends, in an earlier tile or page, with everything before them NaN."""
import pytest
import torch

from tests.test_gpu_paged_attention import Problem, _clean, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def poison(p, window):
    """Tokens before the window are NaN: codes, scales and 16-bit values."""
    for b, n in enumerate(p.lens):
        t = torch.arange(max(0, n - window))
        pg, off = p.table[p.rows[b], t // p.page].long(), t % p.page
        for name in p.names:
            getattr(p, name)[1, pg, :, off] = float("nan") if not p.e4m3 else 0x7F if name in ("k", "v") else 255


@pytest.mark.parametrize("e4m3,dtype", [(False, torch.float16), (False, torch.bfloat16), (True, torch.float16), (True, torch.bfloat16)])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("window", [1, 5, 16, 17, 100, 127, 128, 129, 250, 1000])
def test_window_inside_steps(dev, e4m3, dtype, page, window):  # noqa: F811
    d, hq = (128, 6) if window % 2 else (64, 18)
    p = Problem(dev, [0, 1, 15, 16, 17, 99, 128, 131, 300, 1000, 1003], hq, 2, d, page, dtype, e4m3, seed=window + page)
    poison(p, window)
    o, l = p.run(window=window)
    _clean()
    p.check(o, l, window=window)


@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_before_the_window_are_not_looked_at(dev, e4m3):  # noqa: F811
    """Entries of pages that lie before the window name no page: nothing is reported."""
    p = Problem(dev, [1000, 161], 8, 2, 128, 16, torch.float16, e4m3, seed=5)
    p.table[0, :(1000 - 150) // 16] = -1
    p.table[1, 0] = 10 ** 6                                          # tokens 0 .. 15; the window begins at 16 - 5
    o, l = p.run(window=150)
    _clean(64)
    p.check(o, l, window=150, drop=lambda b, t: (t < 16) if b == 1 else torch.zeros(len(t), dtype=torch.bool))
    p.table[1, 0] = -1
    p.lens[1], p.seq_lens[1], p.seen[1] = 160, 160, [x[:160] for x in p.seen[1]]
    o, l = p.run(window=144)                                        # now at 16
    _clean()
    p.check(o, l, window=144)

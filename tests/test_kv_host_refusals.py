"""Further refusals of the decode-serving calls on the host (no GPU)."""
import ctypes

import pytest
import torch

import block_scaled_quantized_tcgen05_gb300 as q
from tests.test_kv_host import A, B_, CUDA, INVALID, P, SHAPE, _cache, _rope, lib  # noqa: F401


@pytest.mark.parametrize("max_pages", [1 << 60, (1 << 60) + 8, (1 << 62) + 1, (1 << 63) - 1, 1 << 31, (1 << 32) + 8])
def test_page_tables_of_any_size_are_counted(lib, max_pages):  # noqa: F811
    """Pages of 16 tokens: entries whose tokens pass 2^63 are refused like those that pass 2^31."""
    _, kv = _cache(lib)
    rope = _rope(lib)
    for max_seqs in (1, 4):
        table = (P(A), max_pages, max_seqs, max_pages)
        assert lib.qgemm_kv_append(kv, 0, P(A), 512, 128, P(B_), 512, 128, 0, 4, P(A), P(A), *table, rope, None, 0, 0, 0,
                                   None, 0, 0, None) == SHAPE
        assert lib.qgemm_paged_attention(P(A), 1024, 128, 0, 1, 8, kv, 0, *table, P(A), None, P(B_), 1024, 128, None, 0.1, 0,
                                         P(A), 1 << 30, None) == SHAPE
        meta = (kv, *table, P(A), P(A))
        assert lib.qgemm_kv_resize(*meta, P(A), P(A), 2, None) == SHAPE
        assert lib.qgemm_kv_fork(*meta, P(A), P(A), 2, None) == SHAPE
        assert lib.qgemm_kv_compact(*meta, None) == SHAPE
    lib.qgemm_destroy_kv_cache(kv)
    lib.qgemm_destroy_rope(rope)


@pytest.mark.parametrize("args", [
    (128, 0, 1e-300, 1, 1e-20, 0.0, 1.0, 4.0, 1.0),              # 1e295 / 1e-20, past the doubles' end
    (64, 1, 1e4, 1, 1e-320, 0.0, 1.0, 4.0, 1.0),
    (64, 0, 1e4, 2, 1e-320, 64.0, 1.0, 1e6, 1.0),
    (64, 0, 1e4, 0, 1.0, 0.0, 1.0, 4.0, 1e39),                   # a factor that fp32 does not hold
    (64, 0, 1e4, 0, 1.0, 0.0, 1.0, 4.0, -4e38),
])
def test_rope_frequencies_are_finite(lib, args):  # noqa: F811
    out = P()
    assert lib.qgemm_create_rope(ctypes.byref(out), *args) == INVALID, lib.qgemm_last_error_message()
    assert not out.value


@pytest.mark.parametrize("batch,hq,heads,strides", [
    (1, 8, 4, (1020, 128, 1020, 128)), (1, 8, 4, (-3, 128, 7, 128)), (4, 1, 1, (1024, 5, 1024, -1)), (1, 1, 1, (3, 3, 3, 3)),
])
def test_strides_that_are_never_stepped_do_not_count(lib, batch, hq, heads, strides):  # noqa: F811
    """The stride of a dimension of one: a slice of a larger buffer may leave anything there."""
    if torch.cuda.is_available():
        pytest.skip("would launch")
    _, kv = _cache(lib, heads=heads)
    rope = _rope(lib)
    qb, qh, ob, oh = strides
    assert lib.qgemm_paged_attention(P(A), qb, qh, 0, batch, hq, kv, 0, P(A), 8, 4, 8, P(A), None, P(B_), ob, oh, None, 0.1, 0,
                                     P(A), 1 << 30, None) == CUDA, lib.qgemm_last_error_message()
    assert lib.qgemm_rope(P(A), qb, qh, P(B_), ob, oh, 0, batch, hq, 128, P(A), rope, 0, None) == CUDA
    assert lib.qgemm_kv_append(kv, 0, P(A), qb, qh if heads == 1 else 128, P(A), qb, qh if heads == 1 else 128, 0, batch, P(A), P(A),
                               P(A), 8, 4, 8, rope, P(A), qb, qh, hq, P(B_), ob, oh, None) == CUDA
    lib.qgemm_destroy_kv_cache(kv)
    lib.qgemm_destroy_rope(rope)


def _operands(lib, rows=4):  # noqa: F811
    """Host tensors and a view, as the binding takes them."""
    _, handle = _cache(lib)
    kv = q.KVCache(handle.value, q.F16, (2, 8, 4, 16, 128), ())
    x = torch.zeros(rows, 4, 128, dtype=torch.float16)
    return kv, x, torch.zeros(rows, dtype=torch.int32), torch.zeros(rows, 4, dtype=torch.int32)


def test_a_closed_rotation_is_refused(lib):  # noqa: F811
    """Not taken for no rotation."""
    kv, x, i, table = _operands(lib)
    rope = q.qgemm_create_rope(128)
    rope.close()
    with pytest.raises(ValueError, match="closed"):
        q.qgemm_kv_append(kv, 0, x, x, i, i, table, rope=rope, stream=0)
    with pytest.raises(ValueError, match="closed"):
        q.qgemm_rope(x, i, rope, stream=0)


def test_host_tensors_are_refused(lib):  # noqa: F811
    """A tensor in host memory would be an address the GPU cannot read."""
    kv, x, i, table = _operands(lib)
    rope = q.qgemm_create_rope(128)
    lens, refs, w = torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), torch.zeros(1 << 24, dtype=torch.uint8)
    k = torch.zeros(1, 4, 2, 16, 128, dtype=torch.float16)
    for call in (lambda: q.qgemm_rope(x, i, rope, stream=0),
                 lambda: q.qgemm_create_kv_cache(k, k.clone()),
                 lambda: q.qgemm_kv_append(kv, 0, x, x, i, i, table, rope=rope, Q=x, stream=0),
                 lambda: q.qgemm_paged_attention(x, kv, 0, table, lens, x.clone(), workspace=w, stream=0),
                 lambda: q.qgemm_kv_resize(kv, table, lens, refs, i, i, stream=0),
                 lambda: q.qgemm_kv_fork(kv, table, lens, refs, i, i, stream=0),
                 lambda: q.qgemm_kv_compact(kv, table, lens, refs, stream=0),
                 lambda: q.qgemm_kv_copy_pages(kv, i, i, stream=0)):
        with pytest.raises(ValueError, match="device"):
            call()


@pytest.mark.parametrize("max_pages,status", [(1 << 30, CUDA), ((1 << 30) + 1, SHAPE), ((1 << 31) - 1, SHAPE)])
def test_rows_of_more_entries_than_a_cache_has_pages(lib, max_pages, status):  # noqa: F811
    """Pages of one token: the kernels step through a row's entries in 32 bits, up to a thousand past its end."""
    if status == CUDA and torch.cuda.is_available():
        pytest.skip("would launch")
    got, kv = _cache(lib, layers=1, heads=1, page=1, st=(0, 256, 256, 256))
    assert got == 0
    meta = (kv, P(A), max_pages, 1, max_pages, P(A), P(A))
    assert lib.qgemm_kv_resize(*meta, P(A), P(A), 2, None) == status
    assert lib.qgemm_kv_fork(*meta, P(A), P(A), 2, None) == status
    assert lib.qgemm_kv_compact(*meta, None) == status
    lib.qgemm_destroy_kv_cache(kv)

// kv_internal.h -- host-side internals of the paged key-value cache calls.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "qgemm.h"
#include "qgemm_internal.h"

// The view behind qgemm_kv_cache: borrowed device pointers of the two planes and their scales.
// Strides in bytes: layer, page, head, token.
struct qgemm_kv_cache {
    int32_t dtype;
    int64_t layers, pages, heads, page_size, d;
    uint8_t *k, *v;
    int64_t st[4];
    uint8_t *ks, *vs;      // null unless the data is E4M3
    int64_t sst[4];
    int64_t extent, sextent;   // bytes from a plane's base to the end of its last row
    int64_t unit, sunit;       // the largest power of two in every page, head and token stride, bytes
    bool near;                 // offsets of a layer's rows are fewer than 2^32 units
};

// Rotary frequencies: pair i of a head turns by freq[i] / 2^64 of a full turn per position.
struct qgemm_rotation {
    int32_t rot_dim;
    int32_t interleaved;
    float mscale;
    uint64_t freq[128];
};

namespace qgi {

// Bits of the device error word (beside the timeout bits): an index read from device memory (a
// page-table entry, a sequence number, a position) was out of range and what it named was
// skipped; a page operation found too few free pages.
constexpr unsigned ERR_INDEX = 64u;
constexpr unsigned ERR_PAGES = 128u;

// One side of an elementwise pass over [token, head, d] rows, strides in elements.
struct RopeSide {
    const void *x;
    void *y;
    int64_t xt, xh, yt, yh;
    int32_t heads;
};

struct AppendArgs {
    int32_t T;               // tokens
    int32_t d;
    int32_t bf16;            // 16-bit type of the activations
    RopeSide q;              // rotated into y (heads == 0: none)
    const void *k, *v;       // new keys and values (null: no append)
    int64_t kt, kh, vt, vh;
    const qgemm_kv_cache *kv;
    int64_t layer;
    const int32_t *seqs, *pos, *table;
    int64_t table_stride;
    int32_t max_seqs, max_pages;
    const qgemm_rotation *rope;   // null: no rotation
    int32_t inverse;
};
cudaError_t launch_rope_append(const AppendArgs &a, const LaunchCtx &ctx);

struct PagedAttnArgs {
    const void *q;
    int64_t qb, qh;
    void *o;
    int64_t ob, oh;
    float *lse;
    int32_t bf16;
    int32_t B, hq;
    const qgemm_kv_cache *kv;
    int64_t layer;
    const int32_t *table, *lens, *seqs;
    int64_t table_stride;
    int32_t max_seqs, max_pages;
    int32_t window;          // 0: every cached token
    float scale;
    void *workspace;
};
// Workspace: counters (zero before the first call and after each) and the fp32 partial rows of units
// cut by range boundaries; the same whatever the batch.
size_t paged_attention_workspace(const qgemm_kv_cache *kv, int num_sms);
cudaError_t launch_paged_attention(const PagedAttnArgs &a, const LaunchCtx &ctx);

struct PageArgs {
    const qgemm_kv_cache *kv;
    int32_t *table;
    int64_t table_stride;
    int32_t max_seqs, max_pages;
    int32_t *lens, *refs;
};
cudaError_t launch_kv_resize(const PageArgs &a, const int32_t *seqs, const int32_t *new_lens,
                             int32_t n, const LaunchCtx &ctx);
cudaError_t launch_kv_fork(const PageArgs &a, const int32_t *parents, const int32_t *children,
                           int32_t n, const LaunchCtx &ctx);
cudaError_t launch_kv_compact(const PageArgs &a, const LaunchCtx &ctx);
cudaError_t launch_kv_copy_pages(const qgemm_kv_cache *kv, const int32_t *src, const int32_t *dst,
                                 int32_t n, const LaunchCtx &ctx);

}  // namespace qgi

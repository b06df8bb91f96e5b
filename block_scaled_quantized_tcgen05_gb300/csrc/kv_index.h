// kv_index.h -- index arithmetic of the paged key-value cache: where a token lies, and how the
// tiles of a batch are dealt to CTAs.  Plain C++ (host and device), so that the same lines the
// kernels run can be checked on the CPU.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define KV_HD __host__ __device__ __forceinline__
#else
#define KV_HD static inline
#endif

namespace kvi {

// Where token t of a sequence lies: its page and the row inside the page.  `row` is the
// sequence's page-table row (max_pages entries; max_pages * page_size < 2^31).  False, and nothing
// may be accessed, when t is outside the row or the entry names no page of the cache.
KV_HD bool locate(const int32_t *row, int32_t max_pages, int32_t page_size, int32_t pages,
                  int32_t t, int32_t *page, int32_t *off) {
    if (t < 0) return false;
    const int32_t i = (int32_t)((uint32_t)t / (uint32_t)page_size);
    if (i >= max_pages) return false;
    const int32_t p = row[i];
    *page = p;
    *off = t - i * page_size;
    return p >= 0 && p < pages;
}

// Division of a token number t < 2^31 by the page size as a product and a shift: magic = ceil(2^shift /
// page_size) with shift = 31 + l, 2^(l - 1) < page_size <= 2^l, lies in [2^31, 2^32), and its excess times t
// stays below 2^shift / page_size.
KV_HD void page_divisor(int32_t page_size, uint32_t *magic, uint32_t *shift) {
    uint32_t l = 0;
    while ((int64_t(1) << l) < page_size) ++l;
    *shift = 31 + l;
    *magic = (uint32_t)(((uint64_t(1) << *shift) + (uint64_t)page_size - 1) / (uint64_t)page_size);
}
KV_HD int32_t page_of(uint32_t t, uint32_t magic, uint32_t shift) {
    return (int32_t)(((uint64_t)t * magic) >> shift);
}

// Whether row `row` of page `page`, head `head`, its strides and offset counted in units of `unit` bytes, ends inside
// `extent` bytes and its offset fits the 32 bits a kernel forms it in.  64-bit arithmetic: a sum that wraps fails.
KV_HD bool row_inside(uint32_t page, uint32_t page_stride, uint32_t row, uint32_t row_stride, uint32_t head,
                      uint32_t head_stride, uint32_t unit, uint32_t bytes, int64_t extent) {
    const uint64_t last = 0xFFFFFFFFu;
    const uint64_t p = (uint64_t)page * page_stride, r = (uint64_t)row * row_stride, h = (uint64_t)head * head_stride;
    if (p > last || r > last || h > last || p + r + h > last) return false;
    return (p + r + h) * unit + bytes <= (uint64_t)extent;
}

// Pages that hold n tokens.
KV_HD int32_t pages_of(int32_t n, int32_t page_size) { return n > 0 ? (n - 1) / page_size + 1 : 0; }

// The tokens an attention call reads of a sequence of n tokens: [first, n), the last `window` of
// them (0: all).  n is clamped to what the table row can hold.
KV_HD void seen_range(int32_t len, int32_t capacity, int32_t window, int32_t *first, int32_t *n) {
    int32_t m = len < 0 ? 0 : len;
    if (m > capacity) m = capacity;
    *n = m;
    *first = window > 0 && m > window ? m - window : 0;
}

// Tiles of `tile` tokens a range takes; an empty range still counts as one, whose CTA writes the
// empty row's result.
KV_HD int32_t tiles_of(int32_t tokens, int32_t tile) {
    return tokens > 0 ? (tokens - 1) / tile + 1 : 1;
}

// W tiles dealt to G <= W CTAs in contiguous ranges whose sizes differ by at most one: CTA c
// takes [range_begin(c), range_begin(c + 1)).
KV_HD int64_t range_begin(int64_t W, int64_t G, int64_t c) { return W * c / G; }

// The CTA whose range holds tile x (the largest c with range_begin(c) <= x).
KV_HD int64_t range_owner(int64_t W, int64_t G, int64_t x) { return ((x + 1) * G - 1) / W; }

}  // namespace kvi

// kv_pages.cu -- page operations of the paged key-value cache: growing, truncating and freeing
// sequences, forking them, compacting the cache, copying pages.
//
// The page table, the lengths and the pages' reference counts live in device memory and stay there:
// a decode loop grows, forks and frees without a host read-back.  Sequence s of n tokens holds the
// first ceil(n / page_size) entries of its table row; a page is free when its count is 0, and free
// pages are taken lowest first, in the order of the call's items, so the outcome is a function of
// the inputs alone (atomics only add whole numbers).
//
// Two kernels a call.  The first, one block of 1024 threads, does the bookkeeping: it releases,
// scans what every item needs, scans the reference counts for that many free pages (8192 counts a
// pass, stopping when it has enough) and writes the table.  The second moves the data: a warp
// copies the rows of one (page, layer, plane, head), eight 16-byte loads a lane in flight.  Both are
// launched as programmatic dependents, so the second's blocks are resident when the list of copies is ready.
//
// Bound: the data (HBM, read and write) when pages move, launch latency and the chain of dependent
// table reads when they do not.
#include "kv_common.cuh"

namespace qg {
namespace {

constexpr int META_THREADS = 1024;
constexpr int META_WARPS = META_THREADS / 32;
constexpr int SCAN_K = 8;                       // counts a thread tests in one pass

struct Meta {
    int32_t *table;
    int64_t table_stride;
    int32_t max_seqs, max_pages;
    int32_t *lens, *refs;
    int32_t page_size, pages;
    unsigned *err;
};

// Copies the second kernel makes: `tokens` rows of page src into page dst.
struct Copies {
    int32_t *src, *dst, *tokens;    // tokens null: whole pages
    int32_t *count;                 // null: n
    int32_t n;
};

__device__ __forceinline__ bool good_page(const Meta &m, int32_t p) { return p >= 0 && p < m.pages; }
__device__ __forceinline__ bool good_seq(const Meta &m, int32_t s) { return s >= 0 && s < m.max_seqs; }

// A sequence's length as far as its table row goes.
__device__ __forceinline__ int32_t held_tokens(const Meta &m, int32_t seq) {
    const int32_t n = __ldcg(m.lens + seq);
    if (n < 0 || n > m.max_pages * m.page_size) {
        report_index(m.err);
        return n < 0 ? 0 : m.max_pages * m.page_size;
    }
    return n;
}

// Gives back entries [from, to) of a sequence's row (the whole warp).
__device__ __forceinline__ void release(const Meta &m, int32_t seq, int32_t from, int32_t to, int lane) {
    for (int j = from + lane; j < to; j += 32) {
        int32_t *e = m.table + seq * m.table_stride + j;
        const int32_t page = *e;
        *e = -1;
        if (good_page(m, page)) atomicSub(m.refs + page, 1);
        else report_index(m.err);
    }
}

// Exclusive prefix of each thread's x over the block, and the block's total.
template <class I>
__device__ __forceinline__ I block_prefix(I x, I *s_warp, I *total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    I incl = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const I y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    I w = s_warp[lane];                          // META_WARPS == 32
    I wi = w;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const I y = __shfl_up_sync(0xFFFFFFFFu, wi, o);
        if (lane >= o) wi += y;
    }
    *total = __shfl_sync(0xFFFFFFFFu, wi, 31);
    const I base = __shfl_sync(0xFFFFFFFFu, wi - w, warp);
    __syncthreads();                             // s_warp is free again
    return base + incl - x;
}

// Writes the pages of [from, to) whose count is 0 (want_free) or above, in order, to `list` until
// at least `enough` are found; returns how many were found (those past `enough` may be listed too,
// the list has room for `room`).
__device__ int32_t list_pages(const Meta &m, int32_t from, int32_t to, bool want_free, int32_t enough,
                              int32_t *list, int32_t room, int32_t *s_cnt) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int32_t found = 0;
    for (int32_t base = from; base < to && found < enough; base += SCAN_K * META_THREADS) {
        bool hit[SCAN_K];
        uint32_t votes[SCAN_K];
#pragma unroll
        for (int k = 0; k < SCAN_K; ++k) {
            const int32_t i = base + k * META_THREADS + (int)threadIdx.x;
            hit[k] = i < to && i >= base && (__ldcg(m.refs + i) > 0) != want_free;
        }
#pragma unroll
        for (int k = 0; k < SCAN_K; ++k) {
            votes[k] = __ballot_sync(0xFFFFFFFFu, hit[k]);
            if (lane == 0) s_cnt[k * META_WARPS + warp] = __popc(votes[k]);
        }
        __syncthreads();
        // exclusive prefix over the SCAN_K x META_WARPS counts
        int32_t x = threadIdx.x < SCAN_K * META_WARPS ? s_cnt[threadIdx.x] : 0, total;
        __syncthreads();
        const int32_t pre = block_prefix(x, s_cnt + SCAN_K * META_WARPS, &total);
        if (threadIdx.x < SCAN_K * META_WARPS) s_cnt[threadIdx.x] = pre;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < SCAN_K; ++k) {
            const int32_t at = found + s_cnt[k * META_WARPS + warp] + __popc(votes[k] & ((1u << lane) - 1));
            if (hit[k] && at < room) list[at] = base + k * META_THREADS + (int)threadIdx.x;
        }
        __syncthreads();
        found += total;
    }
    return found;
}

// What item i takes, and what becomes of it.
struct Need {
    int32_t pages;       // free pages it needs
    int32_t copy;        // tokens of a page it has to copy (0: none)
};

// RESIZE: sequence seqs[i] gets new_lens[i] tokens (null: none).  Otherwise a fork: children[i]
// (b) becomes a copy of parents[i] (a).
template <bool RESIZE>
__global__ void __launch_bounds__(META_THREADS, 1)
    update_kernel(const Meta m, const int32_t *a, const int32_t *b, int32_t n, int32_t *offset,
                  int32_t *free_list, const Copies copies) {
    __shared__ int64_t s_warp[META_WARPS];
    __shared__ int32_t s_cnt[SCAN_K * META_WARPS + META_WARPS];
    __shared__ int32_t s_copies;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (threadIdx.x == 0) s_copies = 0;
    griddep_launch_dependents();
    griddep_wait();
    const int32_t capacity = m.max_pages * m.page_size;

    // ---- release: what is cut off, and what the children's slots held
    for (int i = warp; i < n; i += META_WARPS) {
        const int32_t seq = RESIZE ? a[i] : b[i];
        const int32_t len = RESIZE ? (b ? b[i] : 0) : 0;
        const bool ok = good_seq(m, seq) && len >= 0 && len <= capacity && (RESIZE || good_seq(m, a[i]));
        if (!ok) {
            if (lane == 0) report_index(m.err);
            continue;
        }
        const int32_t old = held_tokens(m, seq);
        if (len < old) {
            release(m, seq, kvi::pages_of(len, m.page_size), kvi::pages_of(old, m.page_size), lane);
            __syncwarp();
            if (lane == 0) m.lens[seq] = len;
        }
    }
    __threadfence_block();
    __syncthreads();

    // ---- what each item needs, and where its pages begin in the list of free ones
    auto need_of = [&](int i) {
        Need need = {0, 0};
        if (RESIZE) {
            const int32_t seq = a[i], len = b ? b[i] : 0;
            if (!good_seq(m, seq) || len < 0 || len > capacity) return need;
            const int32_t old = held_tokens(m, seq);
            if (len <= old) return need;
            need.pages = kvi::pages_of(len, m.page_size) - kvi::pages_of(old, m.page_size);
            // a last page that others hold too is not written into: it becomes a copy
            const int32_t tail = old % m.page_size;
            if (tail) {
                const int32_t last = m.table[seq * m.table_stride + old / m.page_size];
                if (good_page(m, last) && __ldcg(m.refs + last) > 1) {
                    need.copy = tail;
                    need.pages += 1;
                }
            }
        } else if (good_seq(m, a[i]) && good_seq(m, b[i])) {
            need.copy = held_tokens(m, a[i]) % m.page_size;
            need.pages = need.copy > 0;
        }
        return need;
    };
    int64_t wanted = 0;
    for (int base = 0; base < n; base += META_THREADS) {
        const int i = base + (int)threadIdx.x;
        Need need = {0, 0};
        if (i < n) need = need_of(i);
        int64_t total;
        const int64_t at = wanted + block_prefix<int64_t>(need.pages, s_warp, &total);
        if (i < n) {
            // the item's needs are fixed here: serving another changes the counts
            offset[3 * i] = (int32_t)(at <= m.pages ? at : m.pages);
            offset[3 * i + 1] = need.pages;
            offset[3 * i + 2] = need.copy;
        }
        wanted += total;
    }
    const int32_t enough = (int32_t)(wanted < m.pages ? wanted : m.pages);
    const int32_t found =
        enough > 0 ? list_pages(m, 0, m.pages, true, enough, free_list, m.pages, s_cnt) : 0;
    __threadfence_block();
    __syncthreads();

    // ---- serve the items
    for (int i = warp; i < n; i += META_WARPS) {
        const int32_t at = offset[3 * i], pages = offset[3 * i + 1], copy = offset[3 * i + 2];
        int32_t src = -1, dst = -1;
        const bool ok = RESIZE ? good_seq(m, a[i]) : good_seq(m, a[i]) && good_seq(m, b[i]);
        const bool served = ok && (pages == 0 || (at <= found && pages <= found - at));
        if (ok && !served && lane == 0) atomicOr(m.err, qgi::ERR_PAGES);
        if (served) {
            if (RESIZE) {
                const int32_t seq = a[i], len = b ? b[i] : 0;
                if (len >= 0 && len <= capacity) {
                    const int32_t old = held_tokens(m, seq);
                    int32_t *row = m.table + seq * m.table_stride;
                    if (len > old) {
                        const int32_t have = kvi::pages_of(old, m.page_size);
                        const int first = copy > 0 ? 1 : 0;
                        for (int j = lane; j < pages - first; j += 32) {
                            const int32_t page = free_list[at + first + j];
                            row[have + j] = page;
                            m.refs[page] = 1;
                        }
                        if (first) {
                            src = row[have - 1];
                            dst = free_list[at];
                            __syncwarp();
                            if (lane == 0) {
                                row[have - 1] = dst;
                                m.refs[dst] = 1;
                                atomicSub(m.refs + src, 1);
                            }
                        }
                        __syncwarp();
                        if (lane == 0) m.lens[seq] = len;
                    }
                }
            } else {
                const int32_t parent = a[i], child = b[i], len = held_tokens(m, parent);
                const int32_t *from = m.table + parent * m.table_stride;
                int32_t *row = m.table + child * m.table_stride;
                const int32_t full = len / m.page_size;
                for (int j = lane; j < full; j += 32) {
                    const int32_t page = from[j];
                    row[j] = page;
                    if (good_page(m, page)) atomicAdd(m.refs + page, 1);
                    else report_index(m.err);
                }
                if (copy > 0 && pages > 0) {
                    src = from[full];
                    dst = free_list[at];
                    if (lane == 0) {
                        row[full] = dst;
                        m.refs[dst] = 1;
                    }
                }
                if (lane == 0) m.lens[child] = len;
            }
        }
        if (dst >= 0 && lane == 0) {            // the copies' order does not matter
            const int32_t x = atomicAdd(&s_copies, 1);
            copies.src[x] = src;
            copies.dst[x] = dst;
            copies.tokens[x] = copy;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) *copies.count = s_copies;
}

// Compaction: with U pages in use, those at U and above go to the free ones below U, both in order.
// map[page] is the new place of a page at U or above; *used receives U.
__global__ void __launch_bounds__(META_THREADS, 1)
    compact_kernel(const Meta m, int32_t *map, int32_t *used, const Copies copies) {
    __shared__ int32_t s_warp[META_WARPS];
    __shared__ int32_t s_cnt[SCAN_K * META_WARPS + META_WARPS];
    griddep_launch_dependents();
    griddep_wait();
    int32_t mine = 0, U;
#pragma unroll 8
    for (int i = threadIdx.x; i < m.pages; i += META_THREADS) mine += __ldcg(m.refs + i) > 0;
    block_prefix(mine, s_warp, &U);
    // an entry that names a page nobody counts stays as it is
    for (int i = U + (int)threadIdx.x; i < m.pages; i += META_THREADS) map[i] = i;
    const int32_t holes = list_pages(m, 0, U, true, m.pages, copies.dst, m.pages, s_cnt);
    const int32_t movers = list_pages(m, U, m.pages, false, m.pages, copies.src, m.pages, s_cnt);
    const int32_t n = min(holes, movers);        // equal: U counts the pages in use
    __threadfence_block();
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += META_THREADS) {
        const int32_t from = copies.src[j], to = copies.dst[j];
        map[from] = to;
        m.refs[to] = __ldcg(m.refs + from);
        m.refs[from] = 0;
    }
    if (threadIdx.x == 0) {
        *used = U;
        *copies.count = n;
    }
}

struct Plane {
    uint8_t *base[4];                            // keys, values, their scales
    int64_t layer, page, head, token;
    int64_t slayer, spage, shead, stoken;
    int64_t extent, sextent;
    int32_t layers, heads, rowb, page_size, pages;
    bool scaled;
};

// Copies one (page, layer, plane, head) a warp; REMAP: also replaces the moved pages in the table.
constexpr int COPY_THREADS = 512;
constexpr int REMAP_TILE = COPY_THREADS;

template <bool REMAP>
__global__ void __launch_bounds__(COPY_THREADS)
    copy_kernel(const __grid_constant__ Plane pl, const Copies c, const Meta m, const int32_t *map,
                const int32_t *used, unsigned *err) {
    const int lane = threadIdx.x % 32;
    griddep_launch_dependents();
    griddep_wait();
    if (REMAP) {
        const int32_t U = *used;
        const int per_row = (m.max_pages + REMAP_TILE - 1) / REMAP_TILE;
        for (int64_t x = blockIdx.x; x < (int64_t)m.max_seqs * per_row; x += gridDim.x) {
            const int32_t seq = (int32_t)(x / per_row);
            const int32_t j = (int32_t)(x % per_row) * REMAP_TILE + (int)threadIdx.x;
            const int32_t len = m.lens[seq];
            if (len <= 0 || j >= m.max_pages || j >= kvi::pages_of(len, m.page_size)) continue;
            int32_t *e = m.table + seq * m.table_stride + j;
            const int32_t page = *e;
            if (!good_page(m, page)) report_index(err);
            else if (page >= U) *e = map[page];
        }
    }
    const int32_t n = c.count ? *c.count : c.n;
    const int64_t jobs = (int64_t)n * pl.layers * 2 * pl.heads;
    const int64_t warps = (int64_t)gridDim.x * (COPY_THREADS / 32);
    const int cpr = pl.rowb / 16;                // 16-byte pieces of a row
    for (int64_t job = (int64_t)blockIdx.x * (COPY_THREADS / 32) + threadIdx.x / 32; job < jobs;
         job += warps) {
        const int32_t head = (int32_t)(job % pl.heads);
        int64_t rest = job / pl.heads;
        const int plane = (int)(rest & 1);
        rest >>= 1;
        const int32_t layer = (int32_t)(rest % pl.layers), item = (int32_t)(rest / pl.layers);
        const int32_t src = c.src[item], dst = c.dst[item];
        const int32_t tokens = c.tokens ? c.tokens[item] : pl.page_size;
        if (tokens <= 0) continue;
        if (src < 0 || src >= pl.pages || dst < 0 || dst >= pl.pages) {
            if (lane == 0) report_index(err);
            continue;
        }
        if (src == dst) continue;
        const int64_t at = layer * pl.layer + head * pl.head;
        const uint8_t *from = pl.base[plane] + at + src * pl.page;
        uint8_t *to = pl.base[plane] + at + dst * pl.page;
        [[maybe_unused]] const int64_t last = at + (tokens - 1) * pl.token + pl.rowb;
        if (!QG_IN_BOUNDS(err, at >= 0 && last + src * pl.page <= pl.extent &&
                                   last + dst * pl.page <= pl.extent))
            continue;
        const bool dense = pl.token == pl.rowb;
        const int pieces = tokens * cpr;
        constexpr int K = 8;
        for (int base = lane; base < pieces; base += 32 * K) {
            uint4 v[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int x = base + 32 * k;
                if (x < pieces) {
                    const int64_t o = dense ? (int64_t)x * 16 : x / cpr * pl.token + x % cpr * 16;
                    v[k] = __ldcs(reinterpret_cast<const uint4 *>(from + o));
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int x = base + 32 * k;
                if (x < pieces) {
                    const int64_t o = dense ? (int64_t)x * 16 : x / cpr * pl.token + x % cpr * 16;
                    *reinterpret_cast<uint4 *>(to + o) = v[k];
                }
            }
        }
        if (pl.scaled) {
            const int64_t sat = layer * pl.slayer + head * pl.shead;
            const uint8_t *sf = pl.base[2 + plane] + sat + src * pl.spage;
            uint8_t *st = pl.base[2 + plane] + sat + dst * pl.spage;
            for (int t = lane; t < tokens; t += 32)
                for (int w = 0; w < pl.rowb; w += 128)       // 4 scale bytes every 128 elements
                    *reinterpret_cast<uint32_t *>(st + t * pl.stoken + w / 32) =
                        *reinterpret_cast<const uint32_t *>(sf + t * pl.stoken + w / 32);
        }
    }
}

Plane plane_of(const qgemm_kv_cache *c) {
    Plane p = {};
    p.base[0] = c->k;
    p.base[1] = c->v;
    p.base[2] = c->ks;
    p.base[3] = c->vs;
    p.layer = c->st[0];
    p.page = c->st[1];
    p.head = c->st[2];
    p.token = c->st[3];
    p.slayer = c->sst[0];
    p.spage = c->sst[1];
    p.shead = c->sst[2];
    p.stoken = c->sst[3];
    p.extent = c->extent;
    p.sextent = c->sextent;
    p.layers = (int32_t)c->layers;
    p.heads = (int32_t)c->heads;
    p.scaled = c->dtype == QGEMM_E4M3;
    p.rowb = (int32_t)(c->d * (p.scaled ? 1 : 2));
    p.page_size = (int32_t)c->page_size;
    p.pages = (int32_t)c->pages;
    return p;
}

Meta meta_of(const qgi::PageArgs &a, const qgi::LaunchCtx &ctx) {
    Meta m = {};
    m.table = a.table;
    m.table_stride = a.table_stride;
    m.max_seqs = a.max_seqs;
    m.max_pages = a.max_pages;
    m.lens = a.lens;
    m.refs = a.refs;
    m.page_size = (int32_t)a.kv->page_size;
    m.pages = (int32_t)a.kv->pages;
    m.err = ctx.err;
    return m;
}

// The data kernel for at most `items` copies, two blocks an SM.
template <bool REMAP>
cudaError_t launch_copy(const qgemm_kv_cache *kv, const Copies &c, const Meta &m, const int32_t *map,
                        const int32_t *used, int64_t items, const qgi::LaunchCtx &ctx) {
    const int64_t jobs = items * kv->layers * 2 * kv->heads;
    int64_t blocks = (jobs + COPY_THREADS / 32 - 1) / (COPY_THREADS / 32);
    if (blocks > 2 * (int64_t)ctx.num_sms) blocks = 2 * (int64_t)ctx.num_sms;
    if (blocks < 1) blocks = 1;
    return launch_dependent(copy_kernel<REMAP>, dim3((unsigned)blocks), COPY_THREADS, 0, ctx.stream, plane_of(kv), c, m,
                            map, used, ctx.err);
}

template <bool RESIZE>
cudaError_t launch_update(const qgi::PageArgs &a, const int32_t *x, const int32_t *y, int32_t n,
                          const qgi::LaunchCtx &ctx) {
    const Meta m = meta_of(a, ctx);
    void *scratch = nullptr;
    cudaError_t e = qgi::scratch_alloc(sizeof(int32_t) * (6 * (size_t)n + 1 + (size_t)m.pages), ctx, &scratch);
    if (e != cudaSuccess) return e;
    int32_t *w = static_cast<int32_t *>(scratch);
    Copies c = {};
    c.src = w + 3 * (size_t)n;
    c.dst = w + 4 * (size_t)n;
    c.tokens = w + 5 * (size_t)n;
    c.count = w + 6 * (size_t)n;
    e = launch_dependent(update_kernel<RESIZE>, dim3(1), META_THREADS, 0, ctx.stream, m, x, y, n, w, c.count + 1, c);
    if (e == cudaSuccess) e = launch_copy<false>(a.kv, c, m, nullptr, nullptr, n, ctx);
    const cudaError_t f = qgi::scratch_free(scratch, ctx);
    return e != cudaSuccess ? e : f;
}

}  // namespace
}  // namespace qg

namespace qgi {

cudaError_t launch_kv_resize(const PageArgs &a, const int32_t *seqs, const int32_t *new_lens,
                             int32_t n, const LaunchCtx &ctx) {
    return qg::launch_update<true>(a, seqs, new_lens, n, ctx);
}

cudaError_t launch_kv_fork(const PageArgs &a, const int32_t *parents, const int32_t *children,
                           int32_t n, const LaunchCtx &ctx) {
    return qg::launch_update<false>(a, parents, children, n, ctx);
}

cudaError_t launch_kv_compact(const PageArgs &a, const LaunchCtx &ctx) {
    const qg::Meta m = qg::meta_of(a, ctx);
    void *scratch = nullptr;
    cudaError_t e = scratch_alloc(sizeof(int32_t) * (3 * (size_t)m.pages + 2), ctx, &scratch);
    if (e != cudaSuccess) return e;
    int32_t *w = static_cast<int32_t *>(scratch);
    int32_t *map = w + 2, *used = w;
    qg::Copies c = {};
    c.src = map + m.pages;
    c.dst = c.src + m.pages;
    c.count = w + 1;
    e = qg::launch_dependent(qg::compact_kernel, dim3(1), qg::META_THREADS, 0, ctx.stream, m, map, used, c);
    if (e == cudaSuccess) e = qg::launch_copy<true>(a.kv, c, m, map, used, m.pages, ctx);
    const cudaError_t f = scratch_free(scratch, ctx);
    return e != cudaSuccess ? e : f;
}

cudaError_t launch_kv_copy_pages(const qgemm_kv_cache *kv, const int32_t *src, const int32_t *dst,
                                 int32_t n, const LaunchCtx &ctx) {
    qg::Copies c = {};
    c.src = const_cast<int32_t *>(src);
    c.dst = const_cast<int32_t *>(dst);
    c.n = n;
    return qg::launch_copy<false>(kv, c, qg::Meta{}, nullptr, nullptr, n, ctx);
}

}  // namespace qgi

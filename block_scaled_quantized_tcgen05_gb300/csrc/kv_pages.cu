// kv_pages.cu -- page operations of the paged key-value cache: growing, truncating and freeing
// sequences, forking them, compacting the cache, copying pages.
//
// The page table, the lengths and the pages' reference counts live in device memory and stay there:
// a decode loop grows, forks and frees without a host read-back.  Sequence s of n tokens holds the
// first ceil(n / page_size) entries of its table row; a page is free when its count is 0, and free
// pages are taken lowest first, in the order of the call's items, so the outcome is a function of
// the inputs alone (atomics only add whole numbers).
//
// Two kernels a call.  The first, one block of 512 threads, does the bookkeeping: it releases,
// scans what every item needs, scans the reference counts for that many free pages (4096 counts a
// pass, stopping when it has enough) and writes the table.  It is a chain of dependent reads: what an item
// is, its lengths, its table entries, the counts.  So each is read once, the items and the free pages
// stay in shared memory (up to 1024 of each), and lines needed later are fetched into L2 early.  The second moves the data: a warp
// copies 2 KB of the rows of one (page, layer, plane, head), four 16-byte loads a lane in flight.  Both are
// launched as programmatic dependents, so the second's blocks are resident when the list of copies is ready.
//
// Bound: the data (HBM, read and write) when pages move, launch latency and the chain of dependent
// table reads when they do not.
#include "kv_common.cuh"

namespace qg {
namespace {

constexpr int META_THREADS = 512;
constexpr int META_WARPS = META_THREADS / 32;
constexpr int SCAN_K = 8;                       // counts a thread tests in one pass
constexpr int SCAN = SCAN_K * META_THREADS;     // counts of a pass
static_assert(SCAN_K * META_WARPS == 128, "four counts of hits a lane");
constexpr int CACHED = 1024;                    // items, and listed pages, kept in shared memory

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

__device__ __forceinline__ void fetch_line(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

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
    const I w = lane < META_WARPS ? s_warp[lane] : I(0);
    I wi = w;
#pragma unroll
    for (int o = 1; o < META_WARPS; o *= 2) {
        const I y = __shfl_up_sync(0xFFFFFFFFu, wi, o);
        if (lane >= o) wi += y;
    }
    *total = __shfl_sync(0xFFFFFFFFu, wi, META_WARPS - 1);
    const I base = __shfl_sync(0xFFFFFFFFu, wi - w, warp);
    __syncthreads();                             // s_warp is free again
    return base + incl - x;
}

// Writes the pages of [0, pages) that are free (below `border`) or in use (from it on), in order, to
// `list`, until at least `enough` are found; returns how many (the last pass may list more, up to
// `room`).  s_cnt: two rows of SCAN_K x META_WARPS counts.
__device__ int32_t list_pages(const Meta &m, int32_t border, int32_t enough, int32_t *list, int32_t room,
                              int32_t (*s_cnt)[SCAN_K * META_WARPS]) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int32_t found = 0;
    int pass = 0;
    for (int32_t base = 0; base < m.pages && found < enough; base += SCAN, pass ^= 1) {
        uint32_t votes[SCAN_K];
        int32_t mine[SCAN_K];
#pragma unroll
        for (int k = 0; k < SCAN_K; ++k) {
            const int32_t i = base + k * META_THREADS + (int)threadIdx.x;
            mine[k] = i < m.pages ? __ldcg(m.refs + i) : 0;
        }
#pragma unroll
        for (int k = 0; k < SCAN_K; ++k) {
            const int32_t i = base + k * META_THREADS + (int)threadIdx.x;
            votes[k] = __ballot_sync(0xFFFFFFFFu, i < m.pages && (mine[k] > 0) != (i < border));
            if (lane == 0) s_cnt[pass][k * META_WARPS + warp] = __popc(votes[k]);
        }
        __syncthreads();
        // every warp scans the 128 counts, four a lane; the other row is free for the next pass
        const int4 c = reinterpret_cast<const int4 *>(s_cnt[pass])[lane];
        const int32_t sum = c.x + c.y + c.z + c.w;
        int32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += y;
        }
        const int32_t e0 = incl - sum, e1 = e0 + c.x, e2 = e1 + c.y, e3 = e2 + c.z;
        const int32_t pick = warp % 4 == 0 ? e0 : (warp % 4 == 1 ? e1 : (warp % 4 == 2 ? e2 : e3));
#pragma unroll
        for (int k = 0; k < SCAN_K; ++k) {
            const int32_t before = __shfl_sync(0xFFFFFFFFu, pick, (k * META_WARPS + warp) / 4);
            const int32_t at = found + before + __popc(votes[k] & ((1u << lane) - 1));
            if (((votes[k] >> lane) & 1) && at < room) list[at] = base + k * META_THREADS + (int)threadIdx.x;
        }
        found += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    __syncthreads();
    return found;
}

// An item of a call as the bookkeeping keeps it.
struct Item {
    int32_t seq;         // the sequence that changes (-1: skip the item)
    int32_t from;        // fork: the parent
    int32_t now;         // tokens it holds
    int32_t want;        // tokens it gets
};
struct Need {
    int32_t at;          // its first page in the list of free ones
    int32_t pages;       // free pages it needs
    int32_t copy;        // tokens of a page it has to copy (0: none)
};

// RESIZE: sequence a[i] gets b[i] tokens (b null: none).  Otherwise a fork: b[i] becomes a copy of a[i].
template <bool RESIZE>
__global__ void __launch_bounds__(META_THREADS, 1)
    update_kernel(const Meta m, const int32_t *a, const int32_t *b, int32_t n, Need *far_needs,
                  int32_t *far_list, const Copies copies) {
    __shared__ int64_t s_warp[META_WARPS];
    __shared__ __align__(16) int32_t s_cnt[2][SCAN_K * META_WARPS];
    __shared__ Item s_items[CACHED];
    __shared__ Need s_needs[CACHED];
    __shared__ int32_t s_list[CACHED];
    __shared__ int32_t s_copies;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (threadIdx.x == 0) s_copies = 0;
    griddep_launch_dependents();
    griddep_wait();
    const int32_t capacity = m.max_pages * m.page_size;
    if (threadIdx.x * 32 < min(m.pages, SCAN)) fetch_line(m.refs + threadIdx.x * 32);

    auto read_item = [&](int i) {
        Item x = {-1, 0, 0, 0};
        const int32_t p = a[i], q = RESIZE ? (b ? b[i] : 0) : b[i];
        const bool ok = RESIZE ? good_seq(m, p) && q >= 0 && q <= capacity : good_seq(m, p) && good_seq(m, q);
        if (!ok) {
            report_index(m.err);
            return x;
        }
        x.seq = RESIZE ? p : q;
        x.from = RESIZE ? 0 : p;
        x.now = held_tokens(m, x.seq);
        x.want = RESIZE ? q : held_tokens(m, p);
        return x;
    };
    for (int i = threadIdx.x; i < min(n, CACHED); i += META_THREADS) s_items[i] = read_item(i);
    __syncthreads();
    auto item = [&](int i) { return i < CACHED ? s_items[i] : read_item(i); };

    // ---- release: what is cut off, and what the children's slots held
    for (int i = warp; i < n; i += META_WARPS) {
        const Item x = item(i);
        if (x.seq < 0) continue;
        const int32_t keep = RESIZE ? x.want : 0;
        if (!RESIZE)         // the parent's entries are read below
            for (int j = lane * 32; j < kvi::pages_of(x.want, m.page_size); j += 32 * 32)
                fetch_line(m.table + x.from * m.table_stride + j);
        if (keep < x.now) {
            release(m, x.seq, kvi::pages_of(keep, m.page_size), kvi::pages_of(x.now, m.page_size), lane);
            __syncwarp();
            if (lane == 0) m.lens[x.seq] = keep;
        }
    }
    __threadfence_block();
    __syncthreads();

    // ---- what each item needs, and where its pages begin in the list of free ones; fixed here, since
    // serving one changes the counts
    auto need_of = [&](int i) {
        Need need = {0, 0, 0};
        const Item x = item(i);
        if (x.seq < 0) return need;
        if (RESIZE) {
            if (x.want <= x.now) return need;
            need.pages = kvi::pages_of(x.want, m.page_size) - kvi::pages_of(x.now, m.page_size);
            // a last page that others hold too is not written into: it becomes a copy
            const int32_t tail = x.now % m.page_size;
            if (tail) {
                const int32_t last = m.table[x.seq * m.table_stride + x.now / m.page_size];
                if (!good_page(m, last)) {
                    report_index(m.err);
                } else if (__ldcg(m.refs + last) > 1) {
                    need.copy = tail;
                    need.pages += 1;
                }
            }
        } else {
            // a bad last entry is taken over below as the whole pages' are: a page of the child's own in its place
            // would show what that page held before
            const int32_t tail = x.want % m.page_size;
            if (tail && good_page(m, m.table[x.from * m.table_stride + x.want / m.page_size])) {
                need.copy = tail;
                need.pages = 1;
            }
        }
        return need;
    };
    int64_t wanted = 0;
    for (int base = 0; base < n; base += META_THREADS) {
        const int i = base + (int)threadIdx.x;
        Need need = {0, 0, 0};
        if (i < n) need = need_of(i);
        int64_t total;
        const int64_t at = wanted + block_prefix<int64_t>(need.pages, s_warp, &total);
        need.at = (int32_t)(at <= m.pages ? at : m.pages);
        if (i < n) (i < CACHED ? s_needs[i] : far_needs[i]) = need;
        wanted += total;
    }
    const int32_t enough = (int32_t)(wanted < m.pages ? wanted : m.pages);
    int32_t *list = enough <= CACHED ? s_list : far_list;
    const int32_t found =
        enough > 0 ? list_pages(m, m.pages, enough, list, enough <= CACHED ? CACHED : m.pages, s_cnt) : 0;
    __threadfence_block();
    __syncthreads();

    // ---- serve the items
    for (int i = warp; i < n; i += META_WARPS) {
        const Need need = i < CACHED ? s_needs[i] : far_needs[i];
        Item x = item(i);
        if (x.seq < 0) continue;
        if (need.pages > 0 && (need.at > found || need.pages > found - need.at)) {
            if (lane == 0) atomicOr(m.err, qgi::ERR_PAGES);
            continue;
        }
        int32_t *row = m.table + x.seq * m.table_stride;
        int32_t src = -1, dst = -1;
        if (RESIZE) {
            if (x.want <= x.now) continue;
            const int32_t have = kvi::pages_of(x.now, m.page_size);
            const int first = need.copy > 0 ? 1 : 0;
            for (int j = lane; j < need.pages - first; j += 32) {
                const int32_t page = list[need.at + first + j];
                row[have + j] = page;
                m.refs[page] = 1;
            }
            if (first) {
                src = row[have - 1];
                dst = list[need.at];
                __syncwarp();
                if (lane == 0) {
                    row[have - 1] = dst;
                    m.refs[dst] = 1;
                    atomicSub(m.refs + src, 1);
                }
            }
            __syncwarp();
        } else {
            const int32_t *from = m.table + x.from * m.table_stride;
            const int32_t full = x.want / m.page_size;
            const int32_t shared = need.copy > 0 ? full : kvi::pages_of(x.want, m.page_size);
            if (need.copy > 0) src = from[full];
            for (int j = lane; j < shared; j += 32) {
                const int32_t page = from[j];
                row[j] = page;
                if (good_page(m, page)) atomicAdd(m.refs + page, 1);
                else report_index(m.err);
            }
            if (need.copy > 0) {
                dst = list[need.at];
                if (lane == 0) {
                    row[full] = dst;
                    m.refs[dst] = 1;
                }
            }
        }
        if (lane == 0) {
            m.lens[x.seq] = x.want;
            if (dst >= 0) {                      // the copies' order does not matter
                const int32_t c = atomicAdd(&s_copies, 1);
                copies.src[c] = src;
                copies.dst[c] = dst;
                copies.tokens[c] = need.copy;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) *copies.count = s_copies;
}

// Compaction: with U pages in use, those at U and above go to the free ones below U, both in order.
// map[page] is the new place of a page at U or above; *used receives U.  `list` holds the free ones
// below U, then the pages in use from U on: as many of the one as of the other.
__global__ void __launch_bounds__(META_THREADS, 1)
    compact_kernel(const Meta m, int32_t *map, int32_t *used, int32_t *far_list, const Copies copies) {
    __shared__ int32_t s_warp[META_WARPS];
    __shared__ __align__(16) int32_t s_cnt[2][SCAN_K * META_WARPS];
    __shared__ int32_t s_list[2 * CACHED];
    griddep_launch_dependents();
    griddep_wait();
    int32_t mine = 0, U;
#pragma unroll 8
    for (int i = threadIdx.x; i < m.pages; i += META_THREADS) mine += __ldcg(m.refs + i) > 0;
    block_prefix(mine, s_warp, &U);
    // an entry that names a page nobody counts stays as it is
    for (int i = U + (int)threadIdx.x; i < m.pages; i += META_THREADS) map[i] = i;
    const bool small = m.pages <= 2 * CACHED;
    int32_t *list = small ? s_list : far_list;
    const int32_t n = list_pages(m, U, m.pages + 1, list, m.pages, s_cnt) / 2;
    __threadfence_block();
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += META_THREADS) {
        const int32_t to = list[j], from = list[n + j];
        copies.src[j] = from;
        copies.dst[j] = to;
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

// Copies 2 KB of a (page, layer, plane, head) a warp; REMAP: also replaces the moved pages in the table, 32
// entries a warp, the last warps first (they have the fewest copies).
constexpr int COPY_THREADS = 512;
constexpr int PIECES = 128;                     // 16-byte pieces of a job, four a lane

template <bool REMAP>
__global__ void __launch_bounds__(COPY_THREADS, 2)
    copy_kernel(const __grid_constant__ Plane pl, const Copies c, const Meta m, const int32_t *map,
                const int32_t *used, unsigned *err) {
    const int lane = threadIdx.x % 32;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t warps = (int64_t)gridDim.x * (COPY_THREADS / 32);
    const int64_t warp = (int64_t)blockIdx.x * (COPY_THREADS / 32) + threadIdx.x / 32;
    if (REMAP) {
        const int per_row = (m.max_pages + 31) / 32;
        for (int64_t x = warps - 1 - warp; x < (int64_t)m.max_seqs * per_row; x += warps) {
            const int32_t seq = (int32_t)(x / per_row);
            const int32_t j = (int32_t)(x % per_row) * 32 + lane;
            const int32_t len = m.lens[seq], U = *used;
            if (len <= 0 || j >= m.max_pages || j >= kvi::pages_of(len, m.page_size)) continue;
            int32_t *e = m.table + seq * m.table_stride + j;
            const int32_t page = *e;
            if (!good_page(m, page)) report_index(err);
            else if (page >= U) *e = map[page];
        }
    }
    const int32_t n = c.count ? *c.count : c.n;
    // 2 KB of a (page, layer, plane, head) a job: its 8, 16 or 32 rows from `t0` on.  (256 pages of 8 layers,
    // 554 MB read and written: 92 us at 2 KB, 6.0 TB/s, 98 at 4 KB, whose loads take the registers of a second block.)
    const int cpr = pl.rowb / 16;                // 16-byte pieces of a row
    const int rows = PIECES / cpr, slices = (pl.page_size + rows - 1) / rows;
    const uint32_t strip = 2u * pl.heads * slices, page_jobs = strip * pl.layers;     // below 2^32
    const int64_t jobs = (int64_t)n * page_jobs;
    for (int64_t job = warp; job < jobs; job += warps) {
        const int32_t item = jobs <= 0xFFFFFFFFll ? (int32_t)((uint32_t)job / page_jobs) : (int32_t)(job / page_jobs);
        uint32_t rest = (uint32_t)(job - (int64_t)item * page_jobs);
        const uint32_t layer = rest / strip;
        rest -= layer * strip;
        const uint32_t hp = rest / slices, head = hp >> 1;
        const int plane = (int)(hp & 1);
        const int32_t t0 = (int32_t)(rest - hp * slices) * rows;
        const int32_t src = c.src[item], dst = c.dst[item];
        const int32_t tokens = min((c.tokens ? c.tokens[item] : pl.page_size) - t0, rows);
        if (tokens <= 0) continue;
        if (src < 0 || src >= pl.pages || dst < 0 || dst >= pl.pages) {
            if (lane == 0) report_index(err);
            continue;
        }
        if (src == dst) continue;
        const int64_t at = layer * pl.layer + head * pl.head + t0 * pl.token;
        const uint8_t *from = pl.base[plane] + at + src * pl.page;
        uint8_t *to = pl.base[plane] + at + dst * pl.page;
        [[maybe_unused]] const int64_t last = at + (tokens - 1) * pl.token + pl.rowb;
        if (!QG_IN_BOUNDS(err, at >= 0 && last + src * pl.page <= pl.extent &&
                                   last + dst * pl.page <= pl.extent))
            continue;
        // the row and the place in it of this lane's first piece; the next ones are 32 pieces on
        const int row0 = lane / cpr, step = 32 / cpr;
        const int64_t first = row0 * pl.token + lane % cpr * 16;
        const int pieces = tokens * cpr;
        uint4 v[PIECES / 32];
#pragma unroll
        for (int k = 0; k < PIECES / 32; ++k)
            if (lane + 32 * k < pieces)
                v[k] = __ldcs(reinterpret_cast<const uint4 *>(from + first + k * step * pl.token));
#pragma unroll
        for (int k = 0; k < PIECES / 32; ++k)
            if (lane + 32 * k < pieces) *reinterpret_cast<uint4 *>(to + first + k * step * pl.token) = v[k];
        const int64_t sat = layer * pl.slayer + head * pl.shead + t0 * pl.stoken;
        [[maybe_unused]] const int64_t slast = sat + (tokens - 1) * pl.stoken + 4;
        if (pl.scaled && QG_IN_BOUNDS(err, sat >= 0 && slast + src * pl.spage <= pl.sextent &&
                                               slast + dst * pl.spage <= pl.sextent)) {
            const uint8_t *sf = pl.base[2 + plane] + sat + src * pl.spage;
            uint8_t *st = pl.base[2 + plane] + sat + dst * pl.spage;
            for (int t = lane; t < tokens; t += 32)      // a row's 4 bytes of scales (d <= 128)
                *reinterpret_cast<uint32_t *>(st + t * pl.stoken) =
                    *reinterpret_cast<const uint32_t *>(sf + t * pl.stoken);
        }
    }
}

// whole: the copies are of whole pages, so heads that follow one another are taken as one of all
// their rows.
Plane plane_of(const qgemm_kv_cache *c, bool whole) {
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
    if (whole && c->heads > 1 && p.head == c->page_size * p.token &&
        (!p.scaled || p.shead == c->page_size * p.stoken)) {
        p.page_size *= p.heads;
        p.heads = 1;
    }
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
    const Plane p = plane_of(kv, c.tokens == nullptr);
    const int64_t rows = PIECES / (p.rowb / 16);
    const int64_t jobs = items * p.layers * 2 * p.heads * ((p.page_size + rows - 1) / rows);
    int64_t blocks = (jobs + COPY_THREADS / 32 - 1) / (COPY_THREADS / 32);
    if (blocks > 2 * (int64_t)ctx.num_sms) blocks = 2 * (int64_t)ctx.num_sms;
    if (blocks < 1) blocks = 1;
    return launch_dependent(copy_kernel<REMAP>, dim3((unsigned)blocks), COPY_THREADS, 0, ctx.stream, p, c, m, map, used,
                            ctx.err);
}

template <bool RESIZE>
cudaError_t launch_update(const qgi::PageArgs &a, const int32_t *x, const int32_t *y, int32_t n,
                          const qgi::LaunchCtx &ctx) {
    const Meta m = meta_of(a, ctx);
    void *scratch = nullptr;
    cudaError_t e = qgi::scratch_alloc(sizeof(int32_t) * (6 * (size_t)n + 1 + (size_t)m.pages), ctx, &scratch);
    if (e != cudaSuccess) return e;
    int32_t *w = static_cast<int32_t *>(scratch);
    Copies c = {};               // after the needs (three words each) of the items
    c.src = w + 3 * (size_t)n;
    c.dst = w + 4 * (size_t)n;
    c.tokens = w + 5 * (size_t)n;
    c.count = w + 6 * (size_t)n;
    e = launch_dependent(update_kernel<RESIZE>, dim3(1), META_THREADS, 0, ctx.stream, m, x, y, n,
                         reinterpret_cast<Need *>(w), c.count + 1, c);
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
    cudaError_t e = scratch_alloc(sizeof(int32_t) * (4 * (size_t)m.pages + 2), ctx, &scratch);
    if (e != cudaSuccess) return e;
    int32_t *w = static_cast<int32_t *>(scratch);
    int32_t *map = w + 2, *used = w;
    qg::Copies c = {};
    c.src = map + m.pages;
    c.dst = c.src + m.pages;
    c.count = w + 1;
    e = qg::launch_dependent(qg::compact_kernel, dim3(1), qg::META_THREADS, 0, ctx.stream, m, map, used,
                             c.dst + m.pages, c);
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

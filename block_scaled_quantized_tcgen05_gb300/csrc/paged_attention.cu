// paged_attention.cu -- attention of one new token per sequence over a paged key-value cache.
//
//   o[b, h, :] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale <q[b, h, :], k_j> - max),
//   lse[b, h] = ln sum_j exp(scale <q, k_j>)
//
// over the cached tokens j of sequence b (the last `window` of them); an empty range gives 0 and
// -inf.  The hq / hkv query heads that share a key-value head are computed together, so each cached
// row is read once (per 16 query heads).
//
// Bound: HBM.  A cached key and value of d = 128 take 512 bytes (fp16) or 264 (E4M3) and 4 x 128
// flops per query head, so at 8 heads a key-value head the product needs about an eighth of the
// legacy tensor rate the stream leaves time for.  The matrix unit is therefore used through
// mma.sync with the 16 query rows as its M: scores come out in the layout the second product takes
// its left operand in, so the probabilities never leave the registers, and a tcgen05 tile of 64 or
// 128 rows would be filled to an eighth and send scores and probabilities through TMEM and shared
// memory.
//
// Work.  A unit is (sequence, key-value head, up to 16 of its query heads); its tokens are cut into
// tiles of TILE and the tiles of all units, in order, are dealt to the CTAs in equal contiguous
// ranges, so that ragged lengths load every SM alike whatever the batch.  Each CTA finds its range
// from the lengths on the device (the call is the same for any lengths, so it can be captured).  A
// unit cut by range boundaries leaves fp32 partial rows (max, sum, weighted values) in the
// workspace; the CTA that arrives last merges them in the order of the ranges, so the bits do not
// depend on timing, and nothing waits on another CTA.
//
// Inside a CTA the warps are on their own: each takes STEP tokens of every tile, copies their rows
// into its own ring of shared memory with cp.async (STAGES steps ahead, across unit boundaries: with
// 8 warps about 190 KB an SM are in flight) and keeps its own running maximum, sum and output.
// They meet once per unit, to merge.
//
// Masked places (past the length, outside the window, a bad page) are never read: their rows are
// zero-filled and their scores -inf, so whatever the pages hold there (NaN of an earlier owner) stays
// out.
//
// Precision: scores, softmax and sums in fp32.  P, times 2^15 so that the halves' range is used down to
// 2^-39 of the largest weight, is split into two 16-bit values, hi = p rounded towards zero and lo = rn(p -
// hi) (relative error 2^-21 in fp16, 2^-15 in bf16): with up to 8 query heads the lower 8 of the tile's 16
// rows carry lo at no cost, above 8 it takes a second product.  lo is kept above zero, at 2^-39 of the
// largest weight at least, so that an infinite value stays one (0 x inf and inf - inf would be NaN).  E4M3
// values become the nearest half (bf16) to code * 2^(byte - 127): exact for every block the append writes.
#include <type_traits>

#include "kv_common.cuh"

namespace qg {
namespace {

constexpr int NWARPS = 8;
constexpr int THREADS = 32 * NWARPS;
constexpr int ROWS = 16;                    // query rows of a unit (the mma's M)
constexpr float P_SHIFT = 15.0f;            // P is held times 2^P_SHIFT
constexpr float P_LEAST = 0x1p-24f;         // the smallest half
constexpr float LN2 = 0.69314718055994531f;
constexpr float LOG2E = 1.4426950408889634f;

struct AttnParams {
    const uint8_t *q, *k, *v, *ks, *vs;
    int64_t qb, qh, ob, oh;                 // bytes
    uint8_t *o;
    float *lse;
    int64_t page, head, token, spage, shead, stoken;
    int64_t extent, sextent;
    const int32_t *table, *lens, *seqs;
    int64_t table_stride;
    int32_t B, hq, hkv, group, chunks;      // chunks: units per key-value head
    int32_t max_seqs, max_pages, page_size, pages, window;
    float scale_log2;
    int32_t *counters;
    float *partial;
    unsigned *err;
};

template <class TY_, int D_, bool E4M3_, bool WIDE_>
struct Cfg {
    using TY = TY_;
    static constexpr int D = D_;
    static constexpr bool E4M3 = E4M3_;
    static constexpr bool WIDE = WIDE_;                  // more than 8 query heads a unit
    static constexpr int ROWB = E4M3 ? D : 2 * D;        // bytes of a cached row
    static constexpr int STEP = E4M3 ? 32 : 16;          // tokens of a warp's step
    static constexpr int TILE = STEP * NWARPS;
    static constexpr int CHUNKS = ROWB / 16;             // 16-byte pieces of a row
    static constexpr int PLANE = STEP * ROWB;            // bytes of a step's keys (or values)
    static constexpr int SCALEB = E4M3 ? STEP * 4 : 0;   // scale bytes of a step's keys
    static constexpr int STAGEB = 2 * (PLANE + SCALEB);
    // rows merged at a time: as many as leave room for three stages
    static constexpr int MERGE_ROWS = E4M3 && D == 128 ? 4 : 8;
    static constexpr int MERGEB = NWARPS * MERGE_ROWS * D * 4;
    static constexpr int FIT = (224 * 1024 - MERGEB) / (NWARPS * STAGEB);
    static constexpr int NSTAGES = FIT > 6 ? 6 : FIT;
    static constexpr int SMEM = NWARPS * NSTAGES * STAGEB + MERGEB;
    static constexpr int NT = D / 8;                     // 8-column tiles of the output
    static constexpr int PARTIAL = ROWS * (D + 2);       // floats of a partial
};

__device__ __forceinline__ void mma16816(const bool bf16, float (&c)[4], uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if (bf16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr));
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// 16-byte asynchronous copy past L1; bytes beyond src_bytes (0 or 16) are zero-filled.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(src_bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The 16-byte piece `chunk` of row `row` lies at this piece of the row's place in shared memory.
// 16-bit rows: eight rows of one piece (an ldmatrix) fall into eight bank groups.  8-bit rows: so do
// two rows of four pieces (a key fragment) and four even or four odd rows of two (a value fragment).
template <class C>
__device__ __forceinline__ int swizzle(int row, int chunk) {
    if (!C::E4M3) return chunk ^ (row & (C::CHUNKS < 8 ? C::CHUNKS - 1 : 7));
    if (C::CHUNKS == 8) return chunk ^ ((((row >> 1) & 3) * 2) ^ ((row & 1) * 4));
    return chunk ^ ((row >> 1) & 3);
}

// Two E4M3 codes (low and high byte) times the scales of their blocks, rounded once to the pair of
// 16-bit values.  FAST: both scales are halves (2^-24 .. 2^15), so one half multiply does it.
struct Scale2 {
    uint32_t h2;         // both as halves
    float lo, hi;        // and as fp32 (any byte)
};
__device__ __forceinline__ float scale_f32(uint32_t byte) {
    // 2^(byte - 127): byte 0 is the fp32 subnormal 2^-127, byte 255 NaN
    return __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255 ? 0x7FC00000u : byte << 23));
}
template <class TY, bool FAST>
__device__ __forceinline__ uint32_t decode2(uint16_t codes, const Scale2 &s) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
    if (FAST && !TY::BF16) {
        uint32_t r;
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(s.h2));
        return r;
    }
    const float2 f = TypeF16::unpack(h);
    return TY::pack(f.x * s.lo, f.y * s.hi);
}
template <class TY>
__device__ __forceinline__ Scale2 make_scale(uint32_t lo, uint32_t hi) {
    Scale2 s;
    s.lo = scale_f32(lo);
    s.hi = scale_f32(hi);
    s.h2 = TY::BF16 ? 0u : TypeF16::pack(s.lo, s.hi);
    return s;
}
// Whether a scale byte is outside the halves.
__device__ __forceinline__ bool far_scale(uint32_t byte) { return byte - 103u > 39u; }

// A position in the work: which unit, and which of its tiles.  Held alike by every lane.
struct Cursor {
    int32_t b;            // sequence of the batch
    int32_t hc;           // key-value head * chunks + chunk
    int32_t tile, ntiles; // tile inside the unit, tiles of the unit
    int32_t first, n;     // tokens [first, n)
    int64_t row;          // page-table row (element offset), -1: none
};

__device__ __forceinline__ void seek(Cursor &c, const AttnParams &p, int b, int tile_tokens) {
    c.b = b;
    c.row = -1;
    int32_t len = 0;
    if (b < p.B) {
        const int32_t seq = p.seqs ? p.seqs[b] : b;
        if (seq >= 0 && seq < p.max_seqs) {
            c.row = seq * p.table_stride;
            len = p.lens[seq];
        }
    }
    kvi::seen_range(len, p.max_pages * p.page_size, p.window, &c.first, &c.n);
    c.ntiles = kvi::tiles_of(c.n - c.first, tile_tokens);
}

__device__ __forceinline__ void advance(Cursor &c, const AttnParams &p, int tile_tokens) {
    if (++c.tile < c.ntiles) return;
    c.tile = 0;
    if (++c.hc < p.hkv * p.chunks) return;
    c.hc = 0;
    seek(c, p, c.b + 1, tile_tokens);
}

template <class C>
__global__ void __launch_bounds__(THREADS, 1) paged_attention_kernel(const __grid_constant__ AttnParams p) {
    using TY = typename C::TY;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[NWARPS][ROWS], s_l[NWARPS][ROWS];
    __shared__ int64_t s_scan[NWARPS];
    __shared__ int32_t s_start[4];
    __shared__ uint32_t s_mask[NWARPS][C::NSTAGES];
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, c4 = lane % 4;
    const int units_b = p.hkv * p.chunks;

    // ---- the batch's tiles, and where this CTA's range begins: each thread counts a contiguous
    // piece of the sequences, a scan places the pieces, the piece that holds the start walks to it
    const int per = (p.B + THREADS - 1) / THREADS;
    const int lo_b = min(p.B, tid * per), hi_b = min(p.B, lo_b + per);
    int64_t mine = 0;
    for (int b = lo_b; b < hi_b; ++b) {
        Cursor c;
        seek(c, p, b, C::TILE);
        mine += (int64_t)c.ntiles * units_b;
        if (blockIdx.x == 0) {
            const int32_t seq = p.seqs ? p.seqs[b] : b;
            if (c.row < 0 || p.lens[seq] != c.n) report_index(p.err);
        }
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const int64_t W = total;
    const int64_t G = min((int64_t)gridDim.x, W);
    const int64_t cta = blockIdx.x;
    if (cta >= G) return;
    const int64_t begin = kvi::range_begin(W, G, cta), end = kvi::range_begin(W, G, cta + 1);
    if (begin >= before && begin < before + mine) {
        int64_t at = before;
        for (int b = lo_b; b < hi_b; ++b) {
            Cursor c;
            seek(c, p, b, C::TILE);
            const int64_t n = (int64_t)c.ntiles * units_b;
            if (begin < at + n) {
                s_start[0] = b;
                s_start[1] = (int32_t)((begin - at) / c.ntiles);
                s_start[2] = (int32_t)((begin - at) % c.ntiles);
                break;
            }
            at += n;
        }
    }
    __syncthreads();

    Cursor use;          // the tile being computed
    seek(use, p, s_start[0], C::TILE);
    use.hc = s_start[1];
    use.tile = s_start[2];
    Cursor load = use;   // the tile whose pages are being looked up
    int64_t left = end - begin;             // tiles to compute
    int64_t to_load = left;
    const uint32_t ring = smem_u32(smem) + warp * (C::NSTAGES * C::STAGEB);
    float *merge = reinterpret_cast<float *>(smem + NWARPS * C::NSTAGES * C::STAGEB);

    // ---- page look-up of this warp's tokens of the tile `load` points at, one step ahead of the
    // copies that use it: lane l holds token l's page
    int32_t pg = -1, pt = -1;      // page-table entry and token (-1: none) of the looked-up step
    int32_t phc = 0;               // its head
    auto look_up = [&] {
        pt = -1;
        if (to_load > 0) {
            const int32_t t = load.first + load.tile * C::TILE + warp * C::STEP + lane;
            phc = load.hc;
            if (lane < C::STEP && t < load.n) {
                pt = t;
                pg = p.table[load.row + (uint32_t)t / (uint32_t)p.page_size];
            }
            --to_load;
            if (to_load > 0) advance(load, p, C::TILE);
        }
    };
    // ---- the copies of the looked-up step into ring slot `slot`
    auto issue = [&](int slot) {
        bool ok = pt >= 0;
        int64_t off = 0, soff = 0;
        if (ok) {
            if (pg < 0 || pg >= p.pages) {
                report_index(p.err);
                ok = false;
            } else {
                const int32_t r = pt - (int32_t)((uint32_t)pt / (uint32_t)p.page_size) * p.page_size;
                const int32_t h = phc / p.chunks;
                off = pg * p.page + r * p.token + h * p.head;
                if (C::E4M3) soff = pg * p.spage + r * p.stoken + h * p.shead;
                ok = QG_IN_BOUNDS(p.err, off >= 0 && off + C::ROWB <= p.extent);
                if (!ok) off = soff = 0;
            }
        }
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
        if (lane == 0) s_mask[warp][slot] = mask;
        const uint32_t kd = ring + slot * C::STAGEB, vd = kd + C::PLANE;
        constexpr int RPI = 32 / C::CHUNKS;      // rows an instruction of the warp copies
        const int chunk = lane % C::CHUNKS;
#pragma unroll
        for (int i = 0; i < C::STEP / RPI; ++i) {
            const int r = i * RPI + lane / C::CHUNKS;
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r) + chunk * 16;
            const uint32_t n = (mask >> r) & 1 ? 16 : 0;
            const uint32_t d = r * C::ROWB + swizzle<C>(r, chunk) * 16;
            cp_async_16(kd + d, p.k + o, n);
            cp_async_16(vd + d, p.v + o, n);
        }
        if (C::E4M3) {
            cp_async_4(vd + C::PLANE + lane * 4, p.ks + soff, ok ? 4 : 0);
            cp_async_4(vd + C::PLANE + C::SCALEB + lane * 4, p.vs + soff, ok ? 4 : 0);
        }
    };

    // ---- state of the unit in progress
    uint32_t qa[C::D / 16][4];              // query fragments
    float acc[C::NT][4];
    float m[2], l[2];
    auto start_unit = [&] {
        const int chunk = use.hc % p.chunks, h0 = (use.hc / p.chunks) * p.group + chunk * ROWS;
        const int rows = min(ROWS, p.group - chunk * ROWS);
        const uint8_t *q0 = p.q + use.b * p.qb + (h0 + g) * p.qh;
        const uint8_t *q8 = q0 + 8 * p.qh;
        const bool in0 = g < rows, in8 = C::WIDE && g + 8 < rows;
#pragma unroll
        for (int kk = 0; kk < C::D / 16; ++kk) {
            // 16-bit rows: the fragments ldmatrix gives; 8-bit rows: thread c4 holds 16 consecutive
            // elements of every 64, four for each product, and the queries follow
            const int e = C::E4M3 ? (kk / 4) * 64 + c4 * 16 + (kk % 4) * 4 : kk * 16 + c4 * 2;
            const int e2 = C::E4M3 ? e + 2 : e + 8;
            qa[kk][0] = in0 ? *reinterpret_cast<const uint32_t *>(q0 + 2 * e) : 0;
            qa[kk][2] = in0 ? *reinterpret_cast<const uint32_t *>(q0 + 2 * e2) : 0;
            qa[kk][1] = in8 ? *reinterpret_cast<const uint32_t *>(q8 + 2 * e) : 0;
            qa[kk][3] = in8 ? *reinterpret_cast<const uint32_t *>(q8 + 2 * e2) : 0;
        }
#pragma unroll
        for (int j = 0; j < C::NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
    };

    // ---- one step: scores of STEP tokens, the running softmax, the weighted values
    auto step = [&](int slot, auto fast_tag) {
        [[maybe_unused]] constexpr bool FAST = decltype(fast_tag)::value;
        const uint32_t kd = ring + slot * C::STAGEB, vd = kd + C::PLANE;
        const uint32_t mask = s_mask[warp][slot];
        float s[C::STEP / 8][4];
#pragma unroll
        for (int j = 0; j < C::STEP / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
        if constexpr (!C::E4M3) {
#pragma unroll
            for (int kk = 0; kk < C::D / 16; ++kk) {
                uint32_t b[4];       // lanes 0-15: tokens at piece 2 kk, lanes 16-31: 2 kk + 1
                const int r = lane % 16, ch = 2 * kk + lane / 16;
                ldsm4<false>(kd + r * C::ROWB + swizzle<C>(r, ch) * 16, b);
                mma16816(TY::BF16, s[0], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b[0], b[2]);
                mma16816(TY::BF16, s[1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b[1], b[3]);
            }
        } else {
            const uint32_t ksd = vd + C::PLANE;
#pragma unroll
            for (int j = 0; j < C::STEP / 8; ++j) {
                const int r = 8 * j + g;
#pragma unroll
                for (int hf = 0; hf < C::D / 64; ++hf) {
                    const uint4 w = lds128(kd + r * C::ROWB + swizzle<C>(r, 4 * hf + c4) * 16);
                    const uint32_t byte = lds8(ksd + r * 4 + 2 * hf + c4 / 2);
                    const Scale2 sc = make_scale<TY>(byte, byte);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t b0 = decode2<TY, FAST>(uint16_t(ww[i] & 0xFFFF), sc);
                        const uint32_t b1 = decode2<TY, FAST>(uint16_t(ww[i] >> 16), sc);
                        const int kk = 4 * hf + i;
                        mma16816(TY::BF16, s[j], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b0, b1);
                    }
                }
            }
        }
        // scores in units of log 2; masked ones -inf
        constexpr uint32_t ALL = C::STEP == 32 ? 0xFFFFFFFFu : (1u << (C::STEP % 32)) - 1u;
#pragma unroll
        for (int j = 0; j < C::STEP / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] *= p.scale_log2;
        if (mask != ALL) {
#pragma unroll
            for (int j = 0; j < C::STEP / 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!((mask >> (8 * j + 2 * c4 + (i & 1))) & 1)) s[j][i] = -INFINITY;
        }
        constexpr int NR = C::WIDE ? 2 : 1;
        bool grown = false;
        float nm[2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float x = m[r];
#pragma unroll
            for (int j = 0; j < C::STEP / 8; ++j) x = fmaxf(x, fmaxf(s[j][2 * r], s[j][2 * r + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
            nm[r] = x;
            grown = grown || x > m[r];
        }
        if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                // m = -inf has nothing to scale (its sums are zero)
                const float f = m[r] == -INFINITY ? 0.0f : ex2(m[r] - nm[r]);
                m[r] = nm[r];
                l[r] *= f;
#pragma unroll
                for (int j = 0; j < C::NT; ++j) {
                    acc[j][2 * r] *= f;
                    acc[j][2 * r + 1] *= f;
                    if (!C::WIDE) {
                        acc[j][2] *= f;
                        acc[j][3] *= f;
                    }
                }
            }
        }
        uint32_t hi[C::STEP / 8][2], lo[C::STEP / 8][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float mm = m[r] == -INFINITY ? 0.0f : m[r] - P_SHIFT;
#pragma unroll
            for (int j = 0; j < C::STEP / 8; ++j) {
                const float a = ex2(s[j][2 * r] - mm), b = ex2(s[j][2 * r + 1] - mm);
                l[r] += a + b;
                hi[j][r] = TY::pack_down(a, b);
                const float2 h = TY::unpack(hi[j][r]);
                lo[j][r] = TY::pack(fmaxf(a - h.x, P_LEAST), fmaxf(b - h.y, P_LEAST));
            }
        }
        auto weigh = [&](float (&o)[4], int t, uint32_t b0, uint32_t b1) {
            // tokens 16 t .. 16 t + 15 of the step
            if (C::WIDE) {
                mma16816(TY::BF16, o, hi[2 * t][0], hi[2 * t][1], hi[2 * t + 1][0], hi[2 * t + 1][1], b0, b1);
                mma16816(TY::BF16, o, lo[2 * t][0], lo[2 * t][1], lo[2 * t + 1][0], lo[2 * t + 1][1], b0, b1);
            } else {
                mma16816(TY::BF16, o, hi[2 * t][0], lo[2 * t][0], hi[2 * t + 1][0], lo[2 * t + 1][0], b0, b1);
            }
        };
        if constexpr (!C::E4M3) {
#pragma unroll
            for (int jj = 0; jj < C::NT / 2; ++jj) {
                uint32_t b[4];       // tokens 0-7 and 8-15 of columns 16 jj .. + 7, then of + 8 .. + 15
                const int r = lane % 16, ch = 2 * jj + lane / 16;
                ldsm4<true>(vd + r * C::ROWB + swizzle<C>(r, ch) * 16, b);
                weigh(acc[2 * jj], 0, b[0], b[1]);
                weigh(acc[2 * jj + 1], 0, b[2], b[3]);
            }
        } else {
            // thread (g, c4) takes columns NT g .. NT g + NT - 1 of four tokens: tile j holds column
            // NT n + j in its place n
            const uint32_t vsd = vd + C::PLANE + C::SCALEB;
#pragma unroll
            for (int t = 0; t < C::STEP / 16; ++t) {
                uint32_t w[4][C::NT / 4];
                uint32_t byte[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 16 * t + 2 * c4 + (i & 1) + 8 * (i >> 1);
                    byte[i] = lds8(vsd + r * 4 + (C::NT * g) / 32);
                    if constexpr (C::D == 128) {
                        const uint4 x = lds128(vd + r * C::ROWB + swizzle<C>(r, g) * 16);
                        w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
                    } else {
                        const uint2 x = lds64(vd + r * C::ROWB + swizzle<C>(r, g / 2) * 16 + (g & 1) * 8);
                        w[i][0] = x.x, w[i][1] = x.y;
                    }
                }
                const Scale2 s01 = make_scale<TY>(byte[0], byte[1]), s23 = make_scale<TY>(byte[2], byte[3]);
#pragma unroll
                for (int x = 0; x < C::NT / 4; ++x) {
                    const uint32_t a0 = __byte_perm(w[0][x], w[1][x], 0x5140);
                    const uint32_t a1 = __byte_perm(w[0][x], w[1][x], 0x7362);
                    const uint32_t b0 = __byte_perm(w[2][x], w[3][x], 0x5140);
                    const uint32_t b1 = __byte_perm(w[2][x], w[3][x], 0x7362);
                    weigh(acc[4 * x], t, decode2<TY, FAST>(uint16_t(a0 & 0xFFFF), s01),
                          decode2<TY, FAST>(uint16_t(b0 & 0xFFFF), s23));
                    weigh(acc[4 * x + 1], t, decode2<TY, FAST>(uint16_t(a0 >> 16), s01),
                          decode2<TY, FAST>(uint16_t(b0 >> 16), s23));
                    weigh(acc[4 * x + 2], t, decode2<TY, FAST>(uint16_t(a1 & 0xFFFF), s01),
                          decode2<TY, FAST>(uint16_t(b1 & 0xFFFF), s23));
                    weigh(acc[4 * x + 3], t, decode2<TY, FAST>(uint16_t(a1 >> 16), s01),
                          decode2<TY, FAST>(uint16_t(b1 >> 16), s23));
                }
            }
        }
    };

    // Column of acc[j][i] (i & 1 selects the second of the pair).
    auto column = [&](int j, int i) { return C::E4M3 ? C::NT * (2 * c4 + i) + j : 8 * j + 2 * c4 + i; };

    // Writes four consecutive columns of a finished row.
    auto finish_row = [&](int row, int col, float4 o, float L, float M) {
        const int chunk = use.hc % p.chunks, hkv = use.hc / p.chunks;
        const int in_group = chunk * ROWS + row;
        if (in_group >= p.group) return;
        const int h = hkv * p.group + in_group;
        const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;     // an empty row is 0
        *reinterpret_cast<uint2 *>(p.o + use.b * p.ob + h * p.oh + 2 * col) =
            make_uint2(TY::pack(o.x * inv, o.y * inv), TY::pack(o.z * inv, o.w * inv));
        if (p.lse && col == 0)
            p.lse[(int64_t)use.b * p.hq + h] = L == 0.0f ? -INFINITY : M * LN2 + logf(L);
    };

    // ---- end of the tiles this CTA has of a unit: the warps' rows are merged; a whole unit is
    // written out, a part goes to the workspace
    int64_t unit_at = begin - use.tile;         // the unit's first tile in the whole order
    auto end_unit = [&] {
        const int64_t c_first = kvi::range_owner(W, G, unit_at);
        const int64_t c_last = kvi::range_owner(W, G, unit_at + use.ntiles - 1);
        const bool whole = c_first == c_last;
        float *part = p.partial + (2 * cta + (cta == c_first ? 1 : 0)) * C::PARTIAL;
#pragma unroll
        for (int r = 0; r < (C::WIDE ? 2 : 1); ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
            if (c4 == 0) {
                s_m[warp][g + 8 * r] = m[r] - P_SHIFT;     // the sums are times 2^P_SHIFT
                s_l[warp][g + 8 * r] = l[r];
            }
        }
#pragma unroll
        for (int blk = 0; blk < (C::WIDE ? 16 : 8) / C::MERGE_ROWS; ++blk) {
            const int row0 = blk * C::MERGE_ROWS, half = row0 / 8;
            if (blk) __syncthreads();             // the block before has been read
            if (g >= row0 % 8 && g < row0 % 8 + C::MERGE_ROWS) {
                float *mine_m = merge + (warp * C::MERGE_ROWS + g - row0 % 8) * C::D;
#pragma unroll
                for (int j = 0; j < C::NT; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        mine_m[column(j, i)] =
                            C::WIDE ? acc[j][2 * half + i] : acc[j][i] + acc[j][2 + i];
            }
            __syncthreads();
            // 4 columns a thread
            for (int x = tid; x < C::MERGE_ROWS * C::D / 4; x += THREADS) {
                const int r = x / (C::D / 4), row = row0 + r, col = x % (C::D / 4) * 4;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < NWARPS; ++w) M = fmaxf(M, s_m[w][row]);
                float4 o = make_float4(0, 0, 0, 0);
                float L = 0.0f;
#pragma unroll
                for (int w = 0; w < NWARPS; ++w) {
                    const float mw = s_m[w][row];
                    const float f = mw == -INFINITY ? 0.0f : ex2(mw - M);
                    const float4 a = *reinterpret_cast<const float4 *>(
                        merge + (w * C::MERGE_ROWS + r) * C::D + col);
                    o.x += f * a.x, o.y += f * a.y, o.z += f * a.z, o.w += f * a.w;
                    L += f * s_l[w][row];
                }
                if (whole) {
                    finish_row(row, col, o, L, M);
                } else {
                    *reinterpret_cast<float4 *>(part + row * C::D + col) = o;
                    if (col == 0) {
                        part[ROWS * C::D + row] = M;
                        part[ROWS * C::D + ROWS + row] = L;
                    }
                }
            }
        }
        if (!whole) {
            // the last CTA to arrive merges all parts, in the order of the ranges
            __threadfence();
            __syncthreads();
            const int64_t unit = (int64_t)use.b * units_b + use.hc;
            const int pieces = (int)(c_last - c_first + 1);
            if (tid == 0) {
                const int old = atomicAdd(p.counters + unit, 1);
                s_last = old == pieces - 1;
                if (s_last) p.counters[unit] = 0;          // ready for the next call
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                constexpr int NROWS = C::WIDE ? 16 : 8;
                for (int x = tid; x < NROWS * C::D / 4; x += THREADS) {
                    const int row = x / (C::D / 4), col = x % (C::D / 4) * 4;
                    float M = -INFINITY, L = 0.0f;
                    float4 o = make_float4(0, 0, 0, 0);
                    for (int64_t c = c_first; c <= c_last; ++c) {
                        const float *q = p.partial + (2 * c + (c == c_first ? 1 : 0)) * C::PARTIAL;
                        const float mc = __ldcg(q + ROWS * C::D + row);
                        const float lc = __ldcg(q + ROWS * C::D + ROWS + row);
                        const float4 a = __ldcg(reinterpret_cast<const float4 *>(q + row * C::D + col));
                        const float nM = fmaxf(M, mc);
                        const float fo = M == -INFINITY ? 0.0f : ex2(M - nM);
                        const float fc = mc == -INFINITY ? 0.0f : ex2(mc - nM);
                        M = nM;
                        L = L * fo + lc * fc;
                        o.x = o.x * fo + a.x * fc;
                        o.y = o.y * fo + a.y * fc;
                        o.z = o.z * fo + a.z * fc;
                        o.w = o.w * fo + a.w * fc;
                    }
                    finish_row(row, col, o, L, M);
                }
            }
        }
        __syncthreads();                        // the merge buffer and s_m are free again
    };

    // ---- the loop
    look_up();
#pragma unroll
    for (int i = 0; i < C::NSTAGES - 1; ++i) {
        issue(i);
        cp_commit();
        look_up();
    }
    start_unit();
    int slot = 0, fill = C::NSTAGES - 1;
    while (left > 0) {
        issue(fill);                            // the slot the step before this one has left
        cp_commit();
        look_up();
        cp_wait<C::NSTAGES - 1>();
        __syncwarp();
        if (s_mask[warp][slot] != 0) {
            bool far = false;
            if (C::E4M3 && !TY::BF16) {
                const uint32_t sd = ring + slot * C::STAGEB + 2 * C::PLANE;
                const uint32_t mask = s_mask[warp][slot];
                if ((mask >> lane) & 1) {
#pragma unroll
                    for (int i = 0; i < C::D / 32; ++i)
                        far = far || far_scale(lds8(sd + lane * 4 + i)) ||
                              far_scale(lds8(sd + C::SCALEB + lane * 4 + i));
                }
                far = __any_sync(0xFFFFFFFFu, far);
            }
            if (far) step(slot, std::false_type{});
            else step(slot, std::true_type{});
        }
        __syncwarp();                           // every lane has read the slot
        slot = slot + 1 == C::NSTAGES ? 0 : slot + 1;
        fill = fill + 1 == C::NSTAGES ? 0 : fill + 1;
        --left;
        const bool unit_done = use.tile + 1 == use.ntiles;
        if (unit_done || left == 0) {
            end_unit();
            if (left == 0) break;
            unit_at += use.ntiles;
            advance(use, p, C::TILE);
            start_unit();
        } else {
            ++use.tile;
        }
    }
    cp_wait<0>();
}

template <class C>
cudaError_t launch(const AttnParams &p, int grid, cudaStream_t stream) {
    static_assert(C::SMEM + 3072 <= 227 * 1024, "shared memory");
    static_assert(C::NSTAGES >= 3, "stages");
    cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<C>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    paged_attention_kernel<C><<<grid, THREADS, C::SMEM, stream>>>(p);
    return cudaGetLastError();
}

template <class TY, int D>
cudaError_t launch_cache(const AttnParams &p, bool e4m3, int grid, cudaStream_t stream) {
    const bool wide = p.group > 8;
    if (e4m3) return wide ? launch<Cfg<TY, D, true, true>>(p, grid, stream)
                          : launch<Cfg<TY, D, true, false>>(p, grid, stream);
    return wide ? launch<Cfg<TY, D, false, true>>(p, grid, stream)
                : launch<Cfg<TY, D, false, false>>(p, grid, stream);
}

int64_t chunks_of(int64_t group) { return (group + ROWS - 1) / ROWS; }
size_t counters_bytes(int64_t units) { return (size_t)((units * 4 + 255) / 256 * 256); }
size_t partial_bytes(int64_t d, int num_sms) {
    return ((size_t)num_sms * 2 * ROWS * (size_t)(d + 2) * sizeof(float) + 255) / 256 * 256;
}

}  // namespace
}  // namespace qg

namespace qgi {

size_t paged_attention_workspace(const qgemm_kv_cache *kv, int64_t B, int64_t hq, int num_sms) {
    const int64_t units = B * kv->heads * qg::chunks_of(hq / kv->heads);
    return qg::counters_bytes(units) + qg::partial_bytes(kv->d, num_sms);
}

cudaError_t launch_paged_attention(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    const qgemm_kv_cache *c = a.kv;
    qg::AttnParams p = {};
    p.q = static_cast<const uint8_t *>(a.q);
    p.qb = 2 * a.qb;
    p.qh = 2 * a.qh;
    p.o = static_cast<uint8_t *>(a.o);
    p.ob = 2 * a.ob;
    p.oh = 2 * a.oh;
    p.lse = a.lse;
    p.k = c->k + a.layer * c->st[0];
    p.v = c->v + a.layer * c->st[0];
    p.extent = c->extent - a.layer * c->st[0];
    p.page = c->st[1];
    p.head = c->st[2];
    p.token = c->st[3];
    const bool e4m3 = c->dtype == QGEMM_E4M3;
    if (e4m3) {
        p.ks = c->ks + a.layer * c->sst[0];
        p.vs = c->vs + a.layer * c->sst[0];
        p.sextent = c->sextent - a.layer * c->sst[0];
        p.spage = c->sst[1];
        p.shead = c->sst[2];
        p.stoken = c->sst[3];
    }
    p.table = a.table;
    p.lens = a.lens;
    p.seqs = a.seqs;
    p.table_stride = a.table_stride;
    p.B = a.B;
    p.hq = a.hq;
    p.hkv = (int32_t)c->heads;
    p.group = a.hq / p.hkv;
    p.chunks = (int32_t)qg::chunks_of(p.group);
    p.max_seqs = a.max_seqs;
    p.max_pages = a.max_pages;
    p.page_size = (int32_t)c->page_size;
    p.pages = (int32_t)c->pages;
    p.window = a.window;
    p.scale_log2 = a.scale * qg::LOG2E;
    const int64_t units = (int64_t)a.B * p.hkv * p.chunks;
    p.counters = static_cast<int32_t *>(a.workspace);
    // counters from the front, partial rows at the end: calls of different batches share a workspace
    p.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + a.workspace_bytes / 256 * 256 -
                                          qg::partial_bytes(c->d, ctx.num_sms));
    p.err = ctx.err;
    // no more CTAs than tiles the table rows can hold
    const int64_t cap = (int64_t)a.max_pages * c->page_size;
    const int tile = qg::NWARPS * (e4m3 ? 32 : 16);
    const int64_t most = units * kvi::tiles_of((int32_t)(cap < 0x7FFFFFFF ? cap : 0x7FFFFFFF), tile);
    const int grid = (int)(most < ctx.num_sms ? most : ctx.num_sms);
    if (a.bf16)
        return c->d == 64 ? qg::launch_cache<qg::TypeBF16, 64>(p, e4m3, grid, ctx.stream)
                          : qg::launch_cache<qg::TypeBF16, 128>(p, e4m3, grid, ctx.stream);
    return c->d == 64 ? qg::launch_cache<qg::TypeF16, 64>(p, e4m3, grid, ctx.stream)
                      : qg::launch_cache<qg::TypeF16, 128>(p, e4m3, grid, ctx.stream);
}

}  // namespace qgi

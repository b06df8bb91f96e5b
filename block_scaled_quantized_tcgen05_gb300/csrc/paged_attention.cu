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
// flops per query head, so at 8 heads a key-value head the products need about an eighth of the
// legacy tensor rate the stream leaves time for.  The matrix unit is therefore used through
// mma.sync, with cached rows as the left operand: 16 tokens are the M of the scores S^T = K Q^T, 16
// elements of d that of O^T = V^T P^T, and 8 query heads the N of both, so nothing is padded at 8 heads a
// key-value head; P reaches the second product's layout by a register transpose (movmatrix).  A tcgen05
// tile would take its 128 rows of K and V straight from shared memory, but E4M3 rows have to pass
// through registers to meet their scales, and scores and probabilities would go through TMEM and
// shared memory between the two products of every tile.
//
// Work.  A unit is (sequence, key-value head, up to 16 of its query heads); its tokens are cut into
// tiles of 128, and the tiles of all units, in order, are dealt to the CTAs in equal contiguous
// ranges, so that ragged lengths load every SM alike whatever the batch.  A unit counts EXTRA tiles more
// than it has, for its start and end.  Each CTA finds its range from the lengths on the device (the call
// is the same for any lengths, so it can be captured).  A unit cut by range boundaries leaves fp32 partial
// rows (max, sum, weighted values) in the workspace; of 32 parts in a row the CTA that arrives last merges
// them in the order of the ranges, then of 32 merged ones, so the bits do not depend on timing, and nothing
// waits on another CTA.
//
// Inside a CTA the warps are on their own: each takes 16 tokens of every tile, copies their rows into
// its own ring of shared memory with cp.async (two steps ahead or more, across unit boundaries: about
// 130 KB an SM are in flight) and keeps its own running maximum, sum and output.  They meet once per
// unit, to merge.
//
// Masked places (past the length, outside the window, a bad page) are never read: their rows are
// zero-filled and their scores -inf, so whatever the pages hold there (NaN of an earlier owner) stays
// out.
//
// Precision: scores, softmax and sums in fp32.  P is split into two 16-bit values, hi = p rounded towards zero
// and lo = rn(p - hi) (relative error 2^-21 in fp16, 2^-15 in bf16), and both are multiplied: the matrix unit has
// the time.  Both are kept above zero, so that an infinite value stays one (0 x inf and inf - inf would be NaN).
// Halves of P are times 2^15, so that their range is used down to 2^-39 of the largest weight, the floor (values
// reach 65504: an error of 2.4e-7 a token).  bf16 has fp32's range, and so have its values: a floor of 2^-39 would
// make 1.8 of a vanishing weight's 1e12, and a factor of 2^15 would take the sum past fp32's end from values of
// 1e34 on, so P is as it is there and its floor 2^-126.  E4M3 codes are exact in halves, and are multiplied as
// such; a key block's scale goes onto its part of the score in fp32, and a value becomes the half
// code * 2^(byte - 127), exact, with P in halves too (and no floor: such values are finite).  Where a step's scales
// are not halves, values become the nearest 16-bit value of the activations' type, with P in that type.  bf16
// queries then have both kinds of step on one accumulator: times 2^15 until a value's scale is above 2^60, as it
// is from there on.  (bf16 queries, 128 ragged E4M3 sequences: 133 us; codes brought to bf16 by
// way of fp32 170.)
#include <atomic>
#include <type_traits>

#include "kv_common.cuh"

namespace qg {
namespace {

constexpr int NWARPS = 8;
constexpr int THREADS = 32 * NWARPS;
constexpr int ROWS = 16;                    // query heads of a unit at most
constexpr int STEP = 16;                    // tokens of a warp's step (the scores' M)
constexpr int TILE = STEP * NWARPS;
constexpr float HALF_SHIFT = 15.0f;         // halves of P are times 2^HALF_SHIFT
constexpr uint32_t WIDE = 127 + 60;         // the largest value scale that this factor's sums take
constexpr float LN2 = 0.69314718055994531f;
constexpr float LOG2E = 1.4426950408889634f;

struct AttnParams {
    const uint8_t *q, *k, *v, *ks, *vs;
    int64_t qb, qh, ob, oh;                 // bytes
    uint8_t *o;
    float *lse;
    int64_t extent, sextent;
    const int32_t *table, *lens, *seqs;
    int64_t table_stride;
    int32_t B, hq, hkv, group, chunks;      // chunks: units per key-value head
    int32_t max_seqs, max_pages, page_size, pages, window;
    bool one_page;                          // page_size is a multiple of STEP
    // The cache's strides in units that divide them all, in which a layer's offsets fit 32 bits
    uint32_t unit, page, head, token;
    uint32_t sunit, spage, shead, stoken;
    uint32_t page_magic, page_shift;        // of kvi::page_of
    float scale_log2;
    int32_t *counters;
    int64_t slots;                          // parts there is room for
    float *partial;
    unsigned *err;
};

template <class TY_, int D_, bool E4M3_, int HEADS_>
struct Cfg {
    using TY = TY_;
    static constexpr int D = D_;
    static constexpr bool E4M3 = E4M3_;
    static constexpr int HEADS = HEADS_;                 // query heads of a unit at most: 4, 8 or 16
    static constexpr int NH = HEADS == 16 ? 2 : 1;       // in groups of 8
    // At most 4 heads: columns 4-7 repeat them, and weigh the values with lo where 0-3 do with hi, so that one
    // product does both (128 ragged E4M3 sequences of 4 heads a key-value head: 122 us, with two products 127;
    // 16-bit caches are bound by HBM either way)
    static constexpr bool PACKED = HEADS == 4;
    static constexpr bool SCALED = E4M3 && TY::BF16;     // bf16 queries go into products of halves
    static constexpr float SHIFT = TY::BF16 && !E4M3 ? 0.0f : HALF_SHIFT;    // P is times 2^SHIFT
    static constexpr int ROWB = E4M3 ? D : 2 * D;        // bytes of a cached row
    static constexpr int CHUNKS = ROWB / 16;             // 16-byte pieces of a row
    static constexpr int PLANE = STEP * ROWB;            // bytes of a step's keys (or values)
    static constexpr int SCALEB = E4M3 ? STEP * 4 : 0;   // scale bytes of a step's keys
    static constexpr int STAGEB = 2 * (PLANE + SCALEB);
    // Two CTAs an SM where their registers (8 heads) and three stages each fit; otherwise one
    // (128 ragged E4M3 sequences: 128 us, with one 154; with 16 heads of 64
    // two gain 9 % at many sequences, 35 -> 31 us, and lose as much where few are cut into twice the parts)
    static constexpr bool TWO = NH == 1 && STAGEB <= 4224;
    // heads merged at a time, through the slot of the ring each warp has just read
    static constexpr int MERGE_ROWS = NH == 2 && STAGEB >= 16 * D * 4 ? 16 : 8;
    static_assert(STAGEB >= MERGE_ROWS * D * 4, "a warp's rows fit a slot");
    static constexpr int ROOM = (TWO ? 110 : 224) * 1024;
    static constexpr int FIT = ROOM / (NWARPS * STAGEB);
    static constexpr int NSTAGES = FIT > 6 ? 6 : FIT;
    static constexpr int SMEM = 256 + NWARPS * NSTAGES * STAGEB;
    // What a unit costs beyond its tiles, in tiles (measured, 128 ragged E4M3 sequences: 1 / 2 / 3 extra
    // 132 / 128 / 131 us; 64 ragged fp16 ones 0 / 1 / 2: 123 / 118 / 119)
    static constexpr int EXTRA = ROWB <= 128 ? 2 : 1;
    static constexpr int MT = D / 16;                    // 16-element tiles of the output
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

// The transpose of an 8 x 8 matrix of 16-bit values, a row's pairs over four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
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
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
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

// The factor that takes sums held relative to a maximum of `from` to one of `to`.  Sums of nothing (-inf) count for
// nothing, others for 2^-126 at least, so that an infinite one stays infinite.
__device__ __forceinline__ float rescale(float from, float to) {
    return from == -INFINITY ? 0.0f : fmaxf(ex2(from - to), 0x1p-126f);
}

// The 16-byte piece `chunk` of row `row` lies at this piece of the row's place in shared memory.
// 16-bit rows: eight rows of one piece (an ldmatrix) fall into eight bank groups.  8-bit rows of 128: so
// do four rows of one block's two pieces (a key fragment: rows 0-3 or 4-7, 8 bytes a lane) and four even
// or four odd rows of two pieces (a value fragment).
template <class C>
__device__ __forceinline__ int swizzle(int row, int chunk) {
    if (!C::E4M3) return chunk ^ (row & (C::CHUNKS < 8 ? C::CHUNKS - 1 : 7));
    if (C::CHUNKS == 8) return chunk ^ ((((row >> 1) & 3) * 2) ^ ((row & 1) * 4));
    return chunk ^ ((row >> 1) & 3);
}

// Four E4M3 codes as two pairs of 16-bit values (bytes 0, 1 and 2, 3): exact.
__device__ __forceinline__ void decode4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}
// The scale 2^(byte - 127): byte 0 is the fp32 subnormal 2^-127, byte 255 NaN.  FAST: neither occurs
// (but for the 0 of a masked row, whose codes are 0).
template <bool FAST>
__device__ __forceinline__ float scale_f32(uint32_t byte) {
    if (FAST) return __uint_as_float(byte << 23);
    return __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255 ? 0x7FC00000u : byte << 23));
}
// The scales of a pair of tokens.
struct Scale2 {
    uint32_t h2;         // as halves
    float lo, hi;        // as fp32
};
template <bool FAST>
__device__ __forceinline__ Scale2 make_scale(uint32_t lo, uint32_t hi) {
    Scale2 s;
    s.lo = scale_f32<FAST>(lo);
    s.hi = scale_f32<FAST>(hi);
    s.h2 = FAST ? TypeF16::pack(s.lo, s.hi) : 0u;
    return s;
}
// Four codes times their scales (a pair of tokens' in each half), rounded once to TY.  FAST: TY and the
// scales are halves, so one half multiply does it; through fp32, where the product is exact, otherwise.
template <class TY, bool FAST>
__device__ __forceinline__ void decode4(uint32_t codes, const Scale2 &s, uint32_t &lo, uint32_t &hi) {
    decode4(codes, lo, hi);
    if (FAST) {
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(s.h2));
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(s.h2));
        return;
    }
    const float2 a = TypeF16::unpack(lo), b = TypeF16::unpack(hi);
    lo = TY::pack(a.x * s.lo, a.y * s.hi);
    hi = TY::pack(b.x * s.lo, b.y * s.hi);
}

// A position in the work: which unit, and which of its tiles.  Held alike by every lane.
struct Cursor {
    int32_t rel;          // the tile's place after the range's begin, in tiles and EXTRAs
    int32_t b;            // sequence of the batch
    int32_t h, part;      // key-value head, and which 16 of its query heads
    int32_t tile, ntiles; // tile inside the unit, tiles of the unit
    int32_t first, n;     // tokens [first, n)
    int32_t seq;          // page-table row
    int32_t next_seq, next_len;   // of sequence b + 1, read ahead (-1: none)
};
// What the computing side has to know of a unit, left in shared memory by the look-up.
struct Step {
    int32_t b, hp;        // sequence, key-value head * chunks + part
    int32_t t0;           // place of the unit's first tile after the range's begin (negative: before it)
    int32_t tiles;        // of the unit
};
constexpr int FAN = 32;   // parts of a unit merged at once
constexpr int LEVELS = 2; // FAN^LEVELS parts at most
constexpr int STEPS = 8;  // units looked up and not yet computed, at most

__device__ __forceinline__ int32_t sequence(const AttnParams &p, int b) {
    if (b >= p.B) return -1;
    const int32_t seq = p.seqs ? p.seqs[b] : b;
    return seq >= 0 && seq < p.max_seqs ? seq : -1;
}
// Tokens, and tiles from the 16-token boundary before the first one on.
__device__ __forceinline__ int32_t extent(const AttnParams &p, int32_t len, int32_t *first, int32_t *n) {
    kvi::seen_range(len, p.max_pages * p.page_size, p.window, first, n);
    return kvi::tiles_of(*n - *first / STEP * STEP, TILE);
}
__device__ __forceinline__ void read_ahead(Cursor &c, const AttnParams &p) {
    c.next_seq = sequence(p, c.b + 1);
    c.next_len = c.next_seq >= 0 ? p.lens[c.next_seq] : 0;
}
__device__ __forceinline__ void enter(Cursor &c, const AttnParams &p, int32_t seq, int32_t len) {
    c.seq = max(seq, 0);
    c.ntiles = extent(p, len, &c.first, &c.n);
}
template <class C>
__device__ __forceinline__ void advance(Cursor &c, const AttnParams &p) {
    ++c.rel;
    if (++c.tile < c.ntiles) return;
    c.tile = 0;
    c.rel += C::EXTRA;
    if (++c.part < p.chunks) return;
    c.part = 0;
    if (++c.h < p.hkv) return;
    c.h = 0;
    ++c.b;
    enter(c, p, c.next_seq, c.next_len);
    read_ahead(c, p);
}

// Writes four consecutive elements of a finished row of the unit.
template <class C>
__device__ __forceinline__ void finish_row(const AttnParams &p, const Step &u, int row, int col, float4 o,
                                           float L, float M) {
    using TY = typename C::TY;
    const int hk = u.hp / p.chunks, in_group = (u.hp - hk * p.chunks) * ROWS + row;
    if (in_group >= p.group) return;
    const int h = hk * p.group + in_group;
    const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;     // an empty row is 0
    *reinterpret_cast<uint2 *>(p.o + u.b * p.ob + h * p.oh + 2 * col) =
        make_uint2(TY::pack(o.x * inv, o.y * inv), TY::pack(o.z * inv, o.w * inv));
    if (p.lse && col == 0) p.lse[(int64_t)u.b * p.hq + h] = L == 0.0f ? -INFINITY : M * LN2 + logf(L);
}

// A part of a cut unit is in the workspace (by the whole CTA).  Of FAN parts in a row the CTA that
// arrives last merges them, in the order of the ranges; then, of FAN merged ones, likewise; the last of all
// writes the rows.  Part i of the unit is that of range first + i, in the first slot of its CTA, or in the
// second when it opens the unit.  (32768 tokens of one key-value head, 152 parts: 17 us, and 30 when one
// CTA merges all.  The loops stay rolled: what runs once a call is first fetched, and the same merge
// unrolled by 16 took 1 us more at 6 parts.)
template <class C>
__device__ __forceinline__ void merge_parts(const AttnParams &p, const Step &u, int64_t first, int parts, int mine,
                                         int *s_last) {
    const int tid = threadIdx.x;
    auto slot = [&](int i) { return 2 * (first + i) + (i == 0 ? 1 : 0); };
    int stride = 1;
    for (int level = 0; level < LEVELS; ++level, stride *= FAN) {
        const int i0 = mine - mine % (FAN * stride);
        const int members = min(FAN, (parts - i0 + stride - 1) / stride);
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            int32_t *c = p.counters + (int64_t)level * p.slots + slot(i0);
            const int last = atomicAdd(c, 1) == members - 1;
            if (last) *c = 0;                              // ready for the next call
            *s_last = last;
        }
        __syncthreads();
        if (!*s_last) return;
        __threadfence();
        const bool all = i0 == 0 && members * stride >= parts;
        for (int x = tid; x < C::HEADS * C::D / 4; x += THREADS) {
            const int row = x / (C::D / 4), col = x % (C::D / 4) * 4;
            float M = -INFINITY, L = 0.0f;
            float4 o = make_float4(0, 0, 0, 0);
            const float *ml = p.partial + ROWS * C::D + row;
#pragma unroll 4
            for (int k = 0; k < members; ++k) {            // the loads wait for nothing
                const int64_t at = slot(i0 + k * stride) * C::PARTIAL;
                const float mc = __ldcg(ml + at), lc = __ldcg(ml + at + ROWS);
                const float4 a = __ldcg(reinterpret_cast<const float4 *>(p.partial + at + row * C::D + col));
                const float nM = fmaxf(M, mc);
                const float fo = rescale(M, nM), fc = rescale(mc, nM);
                M = nM;
                L = L * fo + lc * fc;
                o.x = o.x * fo + a.x * fc;
                o.y = o.y * fo + a.y * fc;
                o.z = o.z * fo + a.z * fc;
                o.w = o.w * fo + a.w * fc;
            }
            __syncwarp();                                  // a row's lanes have read its M and L
            if (all) {
                finish_row<C>(p, u, row, col, o, L, M);
            } else {                                       // in the place of the first part
                float *q = p.partial + slot(i0) * C::PARTIAL;
                *reinterpret_cast<float4 *>(q + row * C::D + col) = o;
                if (col == 0) {
                    q[ROWS * C::D + row] = M;
                    q[ROWS * C::D + ROWS + row] = L;
                }
            }
        }
        if (all) return;
        mine = i0;
    }
}

template <class C>
__global__ void __launch_bounds__(THREADS, C::TWO ? 2 : 1)
    paged_attention_kernel(const __grid_constant__ AttnParams p) {
    using TY = typename C::TY;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[NWARPS][ROWS], s_l[NWARPS][ROWS];
    __shared__ int64_t s_scan[NWARPS];
    __shared__ int64_t s_at, s_range[3];     // where the first unit begins; steps in all, ranges, this one's begin
    __shared__ int32_t s_start[3];
    __shared__ uint32_t s_mask[NWARPS][C::NSTAGES];
    __shared__ __align__(16) Step s_step[NWARPS][STEPS];
    __shared__ int s_last;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, c4 = lane % 4;
    const int units_b = p.hkv * p.chunks;

    // ---- the batch's tiles, and where this CTA's range begins: each thread counts a contiguous
    // piece of the sequences, a scan places the pieces, the piece that holds the start walks to it
    const int per = (p.B + THREADS - 1) / THREADS;
    const int lo_b = min(p.B, tid * per), hi_b = min(p.B, lo_b + per);
    int64_t mine = 0;
    int32_t unit_first = 1;              // tiles of a unit of the piece's first sequence
    for (int b = lo_b; b < hi_b; ++b) {
        int32_t first, n;
        const int32_t seq = sequence(p, b), len = seq >= 0 ? p.lens[seq] : 0;
        const int32_t tiles = extent(p, len, &first, &n);
        if (b == lo_b) unit_first = tiles;
        mine += (int64_t)(tiles + C::EXTRA) * units_b;
        if (blockIdx.x == 0 && (seq < 0 || len != n)) report_index(p.err);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int64_t at = incl - mine, W = 0;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) {
        if (w < warp) at += s_scan[w];
        W += s_scan[w];
    }
    const int64_t G = min((int64_t)gridDim.x, W);
    const int64_t cta = blockIdx.x;
    if (cta >= G) return;
    const int64_t begin = kvi::range_begin(W, G, cta), end = kvi::range_begin(W, G, cta + 1);
    if (begin >= at && begin < at + mine) {
        int32_t tiles = unit_first;
        for (int b = lo_b; b < hi_b; ++b) {
            if (b > lo_b) {
                int32_t first, n;
                const int32_t seq = sequence(p, b);
                tiles = extent(p, seq >= 0 ? p.lens[seq] : 0, &first, &n);
            }
            const int64_t n = (int64_t)(tiles + C::EXTRA) * units_b;
            if (begin < at + n) {
                const int32_t hc = (int32_t)((begin - at) / (tiles + C::EXTRA));
                s_start[0] = b;
                s_start[1] = hc;
                s_at = at + (int64_t)hc * (tiles + C::EXTRA);
                break;
            }
            at += n;
        }
    }
    if (tid == 0) {                      // for the ends of units: not worth registers
        s_range[0] = W;
        s_range[1] = G;
        s_range[2] = begin;
    }
    __syncthreads();

    const int32_t span = (int32_t)(end - begin);
    Cursor load;                         // the tile whose pages are being looked up
    load.b = s_start[0];
    load.h = s_start[1] / p.chunks;
    load.part = s_start[1] - load.h * p.chunks;
    {
        const int32_t seq = sequence(p, load.b);
        enter(load, p, seq, seq >= 0 ? p.lens[seq] : 0);
        read_ahead(load, p);
        const int64_t into = begin - s_at - C::EXTRA;      // below 0: inside the unit's EXTRA
        load.tile = (int32_t)max((int64_t)0, into);
        load.rel = (int32_t)max((int64_t)0, -into);
    }
    if (load.rel >= span) return;        // no tile in the range
    // A row's pieces are found by exclusive or from a lane's first address, which takes bases that are
    // multiples of a row (128 bytes for 8-bit rows, whose stages are a multiple of that)
    uint8_t *const base256 = smem + (256 - smem_u32(smem) % 256) % 256;
    const uint32_t ring = smem_u32(base256) + warp * (C::NSTAGES * C::STAGEB);

    // ---- page look-up of this warp's tokens of the tile `load` points at, one step ahead of the
    // copies that use it.  Steps begin at multiples of 16 tokens: with pages of a multiple of 16 tokens
    // a step lies in one page, and every lane holds its entry; otherwise lane l holds token l's (136 us
    // instead of 128 for the ragged E4M3 sequences, 118.4 instead of 117.6 for the fp16 ones).
    struct {
        int32_t pg = -1, pr = 0;         // page-table entry and row inside the page
        int32_t lo = 0, hi = 0;          // rows of the step that are tokens of the range
        int32_t h = 0;                   // its key-value head
    } x;
    int unit = 0;                        // units looked up
    auto look_up = [&](bool opens) {     // the next step of the range; opens: its first
        x.lo = x.hi = 0;
        if (load.rel < span) {
            const int32_t t0 = load.first / STEP * STEP + load.tile * TILE + warp * STEP;
            x.lo = max(load.first - t0, 0);
            x.hi = min(load.n - t0, STEP);
            x.h = load.h;
            const int32_t l = p.one_page ? 0 : lane;
            if (x.lo < x.hi && l < STEP) {
                const int32_t t = t0 + l, i = kvi::page_of((uint32_t)t, p.page_magic, p.page_shift);
                x.pr = t - i * p.page_size;
                // rows before the range's first token may lie in a page of no interest
                if (p.one_page || (l >= x.lo && l < x.hi)) x.pg = p.table[load.seq * p.table_stride + i];
            }
            if (load.tile == 0 || opens) {       // the unit's first tile in the range
                if (lane == 0) {
                    Step st;
                    st.b = load.b;
                    st.hp = load.h * p.chunks + load.part;
                    st.t0 = load.rel - load.tile;
                    st.tiles = load.ntiles;
                    s_step[warp][unit % STEPS] = st;
                }
                ++unit;
            }
            advance<C>(load, p);
        }
    };
    // ---- the copies of the looked-up step into ring slot `slot`
    constexpr int RPI = 32 / C::CHUNKS;          // rows an instruction of the warp copies
    const int chunk = lane % C::CHUNKS, row0 = lane / C::CHUNKS;
    const uint8_t *const lane_k = p.k + chunk * 16, *const lane_v = p.v + chunk * 16;
    const uint32_t lane_row = row0 * p.token;
    const uint32_t lane_to = row0 * C::ROWB + swizzle<C>(row0, chunk) * 16;
    // lanes 0-15: the keys' scale rows, lanes 16-31: the values'
    const uint8_t *const lane_s = lane < STEP ? p.ks : p.vs;
    const uint32_t lane_srow = lane % STEP * p.stoken;
    [[maybe_unused]] auto inside = [&](int32_t pg, int32_t row, int32_t h) {      // the planes, for the debug checks
        return kvi::row_inside(pg, p.page, row, p.token, h, p.head, p.unit, C::ROWB, p.extent) &&
               (!C::E4M3 || kvi::row_inside(pg, p.spage, row, p.stoken, h, p.shead, p.sunit, 4, p.sextent));
    };
    auto issue = [&](int slot) {
        const int32_t pg = x.pg, pr = x.pr, ph = x.h;
        const uint32_t kd = ring + slot * C::STAGEB;
        const bool known = uint32_t(pg) < uint32_t(p.pages);
        uint32_t at = pg * p.page + pr * p.token + ph * p.head;
        const uint32_t sat = pg * p.spage + pr * p.stoken + ph * p.shead;
        if (p.one_page && x.hi - x.lo == STEP && known) {
            // a whole step of one page: rows a token stride apart
            if (QG_IN_BOUNDS(p.err, inside(pg, pr + STEP - 1, ph))) {
                at += lane_row;
#pragma unroll
                for (int i = 0; i < STEP / RPI; ++i) {
                    // swizzle(a + b, c) = swizzle(a, 0) ^ swizzle(b, c) for rows a and b without common bits
                    const uint32_t d = (kd + lane_to) ^ (swizzle<C>(i * RPI, 0) * 16);
                    cp_async_16(d + i * RPI * C::ROWB, lane_k + uint64_t(at) * p.unit, 16);
                    cp_async_16(d + i * RPI * C::ROWB + C::PLANE, lane_v + uint64_t(at) * p.unit, 16);
                    at += RPI * p.token;
                }
                if (C::E4M3)
                    cp_async_4(kd + 2 * C::PLANE + lane * 4, lane_s + uint64_t(sat + lane_srow) * p.sunit, 4);
                if (lane == 0) s_mask[warp][slot] = (1u << STEP) - 1;
                return;
            }
        }
        // lane l: row l's place
        bool ok = lane >= x.lo && lane < x.hi;
        if (ok && !known) report_index(p.err);
        ok = ok && known;
        uint32_t srow = sat;
        if (p.one_page) {
            at += lane * p.token;
            srow += lane_srow;
        }
        ok = ok && QG_IN_BOUNDS(p.err, inside(pg, pr + (p.one_page ? lane : 0), ph));
        if (!ok) at = srow = 0;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok);
        if (lane == 0) s_mask[warp][slot] = mask;
#pragma unroll
        for (int i = 0; i < STEP / RPI; ++i) {
            const int r = i * RPI + row0;
            const uint64_t o = uint64_t(__shfl_sync(0xFFFFFFFFu, at, r)) * p.unit;
            const uint32_t n = (mask >> r) & 1 ? 16 : 0;
            const uint32_t d = (kd + lane_to) ^ (swizzle<C>(i * RPI, 0) * 16);
            cp_async_16(d + i * RPI * C::ROWB, lane_k + o, n);
            cp_async_16(d + i * RPI * C::ROWB + C::PLANE, lane_v + o, n);
        }
        if (C::E4M3) {
            const int r = lane % STEP;
            const uint32_t so = __shfl_sync(0xFFFFFFFFu, srow, r);
            cp_async_4(kd + 2 * C::PLANE + lane * 4, lane_s + uint64_t(so) * p.sunit, (mask >> r) & 1 ? 4 : 0);
        }
    };

    // ---- state of the unit in progress
    uint32_t qb[C::NH][C::D / 16][2];       // query fragments
    float acc[C::NH][C::MT][4];             // rows of d, columns of heads 2 c4, 2 c4 + 1
    float m[C::NH][2], l[C::NH][2];
    float qs[C::NH][2];                     // SCALED: what the scores of heads 2 c4, 2 c4 + 1 are still to be times
    // E4M3.  FAST scales: bytes 112 .. 127 (2^-15 .. 1: blocks of the append up to 512), halves all.  Others take the
    // step through fp32 (all steps so: 172 us instead of 128, bf16 queries 183 instead of 133).
    [[maybe_unused]] constexpr uint32_t HIGH = C::D == 128 ? 0xF0F0F0F0u : 0xF0F0u, FAST_SCALES = HIGH & 0x70707070u;
    // SCALED: what the scales' high bits have to be; nothing is, once the unit has met a value scale above WIDE and its
    // sums hold P as it is (kept as a flag beside the test of the scales it took every step 2 - 5 % longer)
    [[maybe_unused]] uint32_t fast_scales = FAST_SCALES;
    auto wide = [&] { return C::SCALED && fast_scales != FAST_SCALES; };
    auto load_queries = [&](const Step &u) {
        const int h = u.hp / p.chunks, part = u.hp - h * p.chunks;
        const int h0 = h * p.group + part * ROWS, rows = min(ROWS, p.group - part * ROWS);
#pragma unroll
        for (int n = 0; n < C::NH; ++n) {
            const int r = C::PACKED ? g % 4 : 8 * n + g;
            const bool in = r < rows;
            const uint8_t *q = p.q + u.b * p.qb + (h0 + r) * p.qh;
#pragma unroll
            for (int kk = 0; kk < C::D / 16; ++kk) {
                // 16-bit rows: the fragments ldmatrix gives; 8-bit rows: thread c4 holds 8 consecutive
                // elements of every 32, four for each product, and the queries follow
                const int e = C::E4M3 ? (kk / 2) * 32 + c4 * 8 + (kk % 2) * 4 : kk * 16 + c4 * 2;
                const int e2 = C::E4M3 ? e + 2 : e + 8;
                qb[n][kk][0] = in ? *reinterpret_cast<const uint32_t *>(q + 2 * e) : 0;
                qb[n][kk][1] = in ? *reinterpret_cast<const uint32_t *>(q + 2 * e2) : 0;
            }
        }
    };
    // bf16 queries of an E4M3 cache become halves times a power of two that takes the row's largest below
    // 2^15: exact where an element is above 2^-32 of that, off by 2^-40 of it elsewhere
    auto scale_queries = [&] {
        if constexpr (C::SCALED) {
#pragma unroll
            for (int n = 0; n < C::NH; ++n) {
                uint32_t top = 0;            // the largest absolute value's bits, of even and of odd elements
#pragma unroll
                for (int kk = 0; kk < C::D / 16; ++kk)
                    top = __vmaxu2(top, __vmaxu2(qb[n][kk][0] & 0x7FFF7FFFu, qb[n][kk][1] & 0x7FFF7FFFu));
                top = max(top & 0xFFFFu, top >> 16);
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                // 2^k, k = 14 - the largest's exponent, at most 126; infinity and NaN stay what they are
                const uint32_t up = min(268u - (top >> 7), 253u);
                const float f = __uint_as_float(up << 23);
#pragma unroll
                for (int kk = 0; kk < C::D / 16; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 x = TY::unpack(qb[n][kk][i]);
                        qb[n][kk][i] = TypeF16::pack(x.x * f, x.y * f);
                    }
                const float down = __uint_as_float((254u - up) << 23);
#pragma unroll
                for (int i = 0; i < 2; ++i) qs[n][i] = __shfl_sync(0xFFFFFFFFu, down, (2 * c4 + i) * 4);
            }
        }
    };
    auto clear = [&] {
#pragma unroll
        for (int n = 0; n < C::NH; ++n) {
#pragma unroll
            for (int j = 0; j < C::MT; ++j) acc[n][j][0] = acc[n][j][1] = acc[n][j][2] = acc[n][j][3] = 0.0f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }
        fast_scales = FAST_SCALES;
    };
    // the sums so far without their 2^HALF_SHIFT, exactly
    auto widen = [&] {
        fast_scales = ~0u;
#pragma unroll
        for (int n = 0; n < C::NH; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[n][i] *= 0x1p-15f;
#pragma unroll
                for (int j = 0; j < C::MT; ++j) {
                    acc[n][j][i] *= 0x1p-15f;
                    acc[n][j][i + 2] *= 0x1p-15f;
                }
            }
    };

    // Places of this lane's fragments in a step's keys and values: the first piece; the others follow by
    // exclusive or (16-bit rows: the addresses of ldmatrix).
    const int k_row = C::E4M3 ? g : lane % 16, v_row = C::E4M3 ? 2 * c4 : lane % 8 + lane / 16 * 8;
    const uint32_t k_at = k_row * C::ROWB + swizzle<C>(k_row, C::E4M3 ? c4 / 2 : lane / 16) * 16 + (C::E4M3 ? c4 % 2 * 8 : 0);
    const uint32_t v_at =
        v_row * C::ROWB + (!C::E4M3 ? swizzle<C>(v_row, lane / 8 % 2) * 16
                                    : C::D == 128 ? swizzle<C>(v_row, g) * 16 : swizzle<C>(v_row, g / 2) * 16 + g % 2 * 8);

    // ---- one step: scores of 16 tokens, the running softmax, the weighted values
    auto step = [&](int slot, uint32_t mask, auto fast_tag) {
        [[maybe_unused]] constexpr bool FAST = decltype(fast_tag)::value;
        using PT = std::conditional_t<C::E4M3 && FAST, TypeF16, TY>;      // of P and the values
        const uint32_t kd = ring + slot * C::STAGEB, vd = kd + C::PLANE;
        float s[C::NH][4];
#pragma unroll
        for (int n = 0; n < C::NH; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
        if constexpr (!C::E4M3) {
            // two accumulators a group of heads, so that the products' chains are half as long
            float s2[C::NH][4];
#pragma unroll
            for (int n = 0; n < C::NH; ++n) s2[n][0] = s2[n][1] = s2[n][2] = s2[n][3] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < C::D / 16; ++kk) {
                uint32_t a[4];       // tokens 0-7 and 8-15 of piece 2 kk, then of 2 kk + 1
                ldsm4<false>((kd + k_at) ^ (32 * kk), a);
#pragma unroll
                for (int n = 0; n < C::NH; ++n)
                    mma16816(TY::BF16, kk % 2 ? s2[n] : s[n], a[0], a[1], a[2], a[3], qb[n][kk][0], qb[n][kk][1]);
            }
#pragma unroll
            for (int n = 0; n < C::NH; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] += s2[n][i];
        } else {
            // one block of 32 at a time, thread c4 with 8 consecutive bytes of it in two products;
            // the block's scale goes onto its sum, in fp32
            const uint32_t ksd = vd + C::PLANE;
            const uint32_t bx = lds32(ksd + g * 4), by = lds32(ksd + (g + 8) * 4);
#pragma unroll
            for (int blk = 0; blk < C::D / 32; ++blk) {
                const uint32_t at = (kd + k_at) ^ (32 * blk);
                const uint2 x = lds64(at), y = lds64(at + 8 * C::ROWB);       // rows g and g + 8
                const float sx = scale_f32<FAST>((bx >> (8 * blk)) & 255u);
                const float sy = scale_f32<FAST>((by >> (8 * blk)) & 255u);
                uint32_t a[8];
                decode4(x.x, a[0], a[2]);
                decode4(y.x, a[1], a[3]);
                decode4(x.y, a[4], a[6]);
                decode4(y.y, a[5], a[7]);
#pragma unroll
                for (int n = 0; n < C::NH; ++n) {
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma16816(false, part, a[0], a[1], a[2], a[3], qb[n][2 * blk][0], qb[n][2 * blk][1]);
                    mma16816(false, part, a[4], a[5], a[6], a[7], qb[n][2 * blk + 1][0], qb[n][2 * blk + 1][1]);
                    if constexpr (C::SCALED && !FAST)       // first, so that a large scale meets no larger sum
#pragma unroll
                        for (int i = 0; i < 4; ++i) part[i] *= qs[n][i & 1];
                    s[n][0] += sx * part[0];
                    s[n][1] += sx * part[1];
                    s[n][2] += sy * part[2];
                    s[n][3] += sy * part[3];
                }
            }
        }
        // scores in units of log 2, masked ones -inf: [0], [1] of token g, [2], [3] of token g + 8
#pragma unroll
        for (int n = 0; n < C::NH; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (C::SCALED && FAST) s[n][i] *= qs[n][i & 1];
                s[n][i] *= p.scale_log2;
            }
        if (mask != (1u << STEP) - 1) {
            const bool in0 = (mask >> g) & 1, in8 = (mask >> (g + 8)) & 1;
#pragma unroll
            for (int n = 0; n < C::NH; ++n) {
                if (!in0) s[n][0] = s[n][1] = -INFINITY;
                if (!in8) s[n][2] = s[n][3] = -INFINITY;
            }
        }
        bool grown = false;
#pragma unroll
        for (int n = 0; n < C::NH; ++n)
            grown = grown || fmaxf(s[n][0], s[n][2]) > m[n][0] || fmaxf(s[n][1], s[n][3]) > m[n][1];
        if (__any_sync(0xFFFFFFFFu, grown)) {
#pragma unroll
            for (int n = 0; n < C::NH; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = fmaxf(m[n][i], fmaxf(s[n][i], s[n][i + 2]));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                    const float f = rescale(m[n][i], x);
                    m[n][i] = x;
                    l[n][i] *= f;
#pragma unroll
                    for (int j = 0; j < C::MT; ++j) {
                        acc[n][j][i] *= f;
                        acc[n][j][i + 2] *= f;
                    }
                }
        }
        uint32_t hi[C::NH][2], lo[C::NH][2];
#pragma unroll
        for (int n = 0; n < C::NH; ++n) {
            const float shift = !FAST && wide() ? 0.0f : C::SHIFT;
            const float m0 = m[n][0] == -INFINITY ? 0.0f : m[n][0] - shift;
            const float m1 = m[n][1] == -INFINITY ? 0.0f : m[n][1] - shift;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float a = ex2(s[n][2 * i] - m0), b = ex2(s[n][2 * i + 1] - m1);
                l[n][0] += a;
                l[n][1] += b;
                // halves of an E4M3 cache hold no infinity that a zero could meet
                constexpr bool FINITE = C::E4M3 && FAST;
                auto positive = [](float x) {
                    return FINITE ? x : fmaxf(x, PT::BF16 ? 0x1p-126f : 0x1p-24f);
                };
                const uint32_t h = PT::pack_down(positive(a), positive(b));
                const float2 f = PT::unpack(h);
                const uint32_t r = PT::pack(positive(a - f.x), positive(b - f.y));
                hi[n][i] = transpose8(C::PACKED && c4 >= 2 ? r : h);
                if (!C::PACKED) lo[n][i] = transpose8(r);
            }
        }
        auto weigh = [&](int j, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int n = 0; n < C::NH; ++n) {
                mma16816(PT::BF16, acc[n][j], a0, a1, a2, a3, hi[n][0], hi[n][1]);
                mma16816(PT::BF16, acc[n][j], a0, a1, a2, a3, lo[n][0], lo[n][1]);
            }
        };
        if constexpr (!C::E4M3) {
#pragma unroll
            for (int j = 0; j < C::MT; ++j) {
                uint32_t a[4];       // tokens 0-7: elements 16 j .. + 7, + 8 .. + 15; tokens 8-15 likewise
                ldsm4<true>((vd + v_at) ^ (32 * j), a);
                weigh(j, a[0], a[1], a[2], a[3]);
            }
        } else {
            // thread (g, c4) takes elements D / 8 g .. + D / 8 - 1 of four tokens: tile j holds element
            // D / 8 r + 2 j in its row r and the next one in row r + 8
            const uint32_t vsd = vd + C::PLANE + C::SCALEB;
            uint32_t w[4][C::D / 32];
            uint32_t byte[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 2 * c4 + (i & 1) + 8 * (i >> 1);
                byte[i] = lds8(vsd + r * 4 + (C::D / 8 * g) / 32);
                if constexpr (C::D == 128) {
                    const uint4 x = lds128(((vd + v_at) ^ (i & 1 ? swizzle<C>(1, 0) * 16 : 0)) +
                                           ((i & 1) + 8 * (i >> 1)) * C::ROWB);
                    w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
                } else {
                    const uint2 x = lds64(((vd + v_at) ^ (i & 1 ? swizzle<C>(1, 0) * 16 : 0)) +
                                          ((i & 1) + 8 * (i >> 1)) * C::ROWB);
                    w[i][0] = x.x, w[i][1] = x.y;
                }
            }
            const Scale2 s01 = make_scale<FAST>(byte[0], byte[1]), s23 = make_scale<FAST>(byte[2], byte[3]);
#pragma unroll
            for (int x = 0; x < C::D / 32; ++x) {
                uint32_t t[2][4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t a = __byte_perm(w[0][x], w[1][x], y ? 0x7362 : 0x5140);
                    const uint32_t b = __byte_perm(w[2][x], w[3][x], y ? 0x7362 : 0x5140);
                    decode4<PT, FAST>(a, s01, t[y][0], t[y][1]);
                    decode4<PT, FAST>(b, s23, t[y][2], t[y][3]);
                }
#pragma unroll
                for (int n = 0; n < C::NH; ++n) {
                    mma16816(PT::BF16, acc[n][2 * x], t[0][0], t[0][1], t[0][2], t[0][3], hi[n][0], hi[n][1]);
                    mma16816(PT::BF16, acc[n][2 * x + 1], t[1][0], t[1][1], t[1][2], t[1][3], hi[n][0], hi[n][1]);
                    if (C::PACKED) continue;
                    mma16816(PT::BF16, acc[n][2 * x], t[0][0], t[0][1], t[0][2], t[0][3], lo[n][0], lo[n][1]);
                    mma16816(PT::BF16, acc[n][2 * x + 1], t[1][0], t[1][1], t[1][2], t[1][3], lo[n][0], lo[n][1]);
                }
            }
        }
    };

    // Place of 16-byte piece u in a merged row: the four pairs of heads, whose lanes write together, go
    // to different banks.
    auto place = [&](int u, int row) {
        const int pair = (row >> 1) & 3;
        if (!C::E4M3) return u ^ (2 * pair);
        return u ^ (C::D == 128 ? pair : (pair & 1) | ((pair & 2) << 1));
    };

    // ---- end of the tiles this CTA has of a unit: the warps' rows are merged, through the ring's slots
    // that were just read (a buffer of its own leaves room for 2 heads at a time beside two CTAs' rings: the
    // 128 ragged E4M3 sequences took 12 % longer); a whole unit is written out, a part goes to the workspace
    auto end_unit = [&](const Step &u, int slot) {
        const int32_t tiles = u.tiles;
        const bool opens = u.t0 >= 0, whole = opens && u.t0 + tiles <= span;
        // the slot `slot` of each warp's ring, read by the step before and not filled again yet
        auto rows_of = [&](int w) {
            return reinterpret_cast<float *>(base256 + (w * C::NSTAGES + slot) * C::STAGEB);
        };
        // a part lies in the slot of its CTA's range: the second when it opens the unit
        float *part = p.partial + (2 * (int64_t)blockIdx.x + (opens ? 1 : 0)) * C::PARTIAL;
#pragma unroll
        for (int n = 0; n < C::NH; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 4);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 8);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 16);
                if (g == 0) {
                    s_m[warp][8 * n + 2 * c4 + i] = m[n][i] - (wide() ? 0.0f : C::SHIFT);    // what the sums are times
                    s_l[warp][8 * n + 2 * c4 + i] = l[n][i];
                }
            }
#pragma unroll
        for (int blk = 0; blk < 8 * C::NH / C::MERGE_ROWS; ++blk) {
            if (blk) __syncthreads();                     // the block before has been read
#pragma unroll
            for (int n8 = 0; n8 < C::MERGE_ROWS / 8; ++n8) {
                const int n = blk * (C::MERGE_ROWS / 8) + n8;
                float *dst = rows_of(warp) + (8 * n8 + 2 * c4) * C::D;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if constexpr (C::E4M3) {         // D / 8 consecutive elements a lane
#pragma unroll
                        for (int j = 0; j < C::MT; j += 2)
                            *reinterpret_cast<float4 *>(dst + i * C::D + 4 * place((C::D / 8 * g + 2 * j) / 4, 2 * c4)) =
                                make_float4(acc[n][j][i], acc[n][j][i + 2], acc[n][j + 1][i], acc[n][j + 1][i + 2]);
                    } else {
#pragma unroll
                        for (int j = 0; j < C::MT; ++j)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int e = 16 * j + 8 * half + g;
                                dst[i * C::D + 4 * place(e / 4, 2 * c4) + e % 4] = acc[n][j][i + 2 * half];
                            }
                    }
                }
            }
            __syncthreads();
            // 4 elements a thread
            for (int x = tid; x < (C::PACKED ? 4 : C::MERGE_ROWS) * C::D / 4; x += THREADS) {
                const int r = x / (C::D / 4), row = blk * C::MERGE_ROWS + r, col = x % (C::D / 4) * 4;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < NWARPS; ++w) M = fmaxf(M, s_m[w][row]);
                float4 o = make_float4(0, 0, 0, 0);
                float L = 0.0f;
#pragma unroll
                for (int w = 0; w < NWARPS; ++w) {
                    const float mw = s_m[w][row];
                    const float f = rescale(mw, M);
                    const float4 a = *reinterpret_cast<const float4 *>(
                        rows_of(w) + r * C::D + 4 * place(col / 4, row));
                    o.x += f * a.x, o.y += f * a.y, o.z += f * a.z, o.w += f * a.w;
                    if constexpr (C::PACKED) {
                        const float4 b = *reinterpret_cast<const float4 *>(
                            rows_of(w) + (r + 4) * C::D + 4 * place(col / 4, row + 4));
                        o.x += f * b.x, o.y += f * b.y, o.z += f * b.z, o.w += f * b.w;
                    }
                    L += f * s_l[w][row];
                }
                if (whole) {
                    finish_row<C>(p, u, row, col, o, L, M);
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
            const int64_t first = kvi::range_owner(s_range[0], s_range[1], s_range[2] + u.t0);
            const int64_t last = kvi::range_owner(s_range[0], s_range[1], s_range[2] + u.t0 + tiles - 1);
            merge_parts<C>(p, u, first, (int)(last - first + 1), (int)(blockIdx.x - first), &s_last);
        }
        __syncthreads();                        // the slots and s_m are free again
    };

    // ---- the loop
    look_up(true);
    for (int i = 0; i < C::NSTAGES - 1; ++i) {
        issue(i);
        cp_commit();
        look_up(false);
    }
    __syncwarp();
    load_queries(s_step[warp][0]);
    scale_queries();
    clear();
    int slot = 0, fill = C::NSTAGES - 1;
    int at_unit = 0;                     // unit being computed, and how many of its steps are left
    auto left_of = [&](const Step &u) {                  // tiles of the unit that are the range's
        return min(u.tiles + u.t0, span) - max(u.t0, 0);
    };
    int left = left_of(s_step[warp][0]);
#pragma unroll 1
    for (;;) {
        issue(fill);                     // the slot the step before this one has left
        cp_commit();
        look_up(false);
        fill = fill + 1 == C::NSTAGES ? 0 : fill + 1;
        cp_wait<C::NSTAGES - 1>();
        __syncwarp();
        const uint32_t mask = s_mask[warp][slot];
        if (mask != 0) {
            bool far = false;
            if (C::E4M3) {
                const uint32_t w = lds32(ring + slot * C::STAGEB + 2 * C::PLANE + lane * 4);
                far = ((mask >> (lane % STEP)) & 1) && (w & HIGH) != (C::SCALED ? fast_scales : FAST_SCALES);
                far = __any_sync(0xFFFFFFFFu, far);
            }
            if (far) {
                if constexpr (C::SCALED) {
                    if (!wide()) {                      // lanes 16-31: the values' scales, 0 for masked rows
                        const uint32_t w = lds32(ring + slot * C::STAGEB + 2 * C::PLANE + lane * 4);
                        const uint32_t over = __vcmpgtu4(C::D == 128 ? w : w & 0xFFFFu, WIDE * 0x01010101u);
                        if (__any_sync(0xFFFFFFFFu, lane >= STEP && over != 0)) widen();
                    }
                }
                step(slot, mask, std::false_type{});
            } else {
                step(slot, mask, std::true_type{});
            }
        }
        __syncwarp();                           // every lane has read the slot
        if (--left == 0) {
            const Step done = s_step[warp][at_unit % STEPS];
            const bool more = done.t0 + done.tiles + C::EXTRA < span;
            ++at_unit;
            if (more) load_queries(s_step[warp][at_unit % STEPS]);   // in flight while the warps merge
            end_unit(done, slot);
            if (!more) break;
            scale_queries();
            clear();
            left = left_of(s_step[warp][at_unit % STEPS]);
        }
        slot = slot + 1 == C::NSTAGES ? 0 : slot + 1;
    }
    cp_wait<0>();
}

template <class C>
cudaError_t launch(const AttnParams &p, int64_t most, const qgi::LaunchCtx &ctx) {
    static_assert(C::SMEM + 2560 <= (C::TWO ? 113 : 227) * 1024, "shared memory");
    static_assert(C::NSTAGES >= 3, "stages");
    // the attribute stays with the device's context: set once on each device
    static std::atomic<uint64_t> ready{0};
    if (!(ready.load(std::memory_order_relaxed) >> ctx.device & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<C>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        ready.fetch_or(uint64_t(1) << ctx.device, std::memory_order_relaxed);
    }
    const int64_t room = (int64_t)ctx.num_sms * (C::TWO ? 2 : 1);
    return launch_dependent(paged_attention_kernel<C>, dim3((unsigned)(most < room ? most : room)), THREADS, C::SMEM,
                            ctx.stream, p);
}

template <class TY, int D>
cudaError_t launch_cache(const AttnParams &p, bool e4m3, int64_t most, const qgi::LaunchCtx &ctx) {
    const bool wide = p.group > 8;
    if (!e4m3) return wide ? launch<Cfg<TY, D, false, 16>>(p, most, ctx) : launch<Cfg<TY, D, false, 8>>(p, most, ctx);
    if (p.group <= 4) return launch<Cfg<TY, D, true, 4>>(p, most, ctx);
    return wide ? launch<Cfg<TY, D, true, 16>>(p, most, ctx) : launch<Cfg<TY, D, true, 8>>(p, most, ctx);
}

int64_t chunks_of(int64_t group) { return (group + ROWS - 1) / ROWS; }
// Parts that can wait at once: two a CTA (the unit that began before its range, the one that goes on
// after it), up to two CTAs an SM.
int64_t slots_of(int num_sms) { return 4 * (int64_t)num_sms; }
size_t counters_bytes(int num_sms) {
    return (size_t)((LEVELS * slots_of(num_sms) * sizeof(int32_t) + 255) / 256 * 256);
}

}  // namespace
}  // namespace qg

namespace qgi {

size_t paged_attention_workspace(const qgemm_kv_cache *kv, int num_sms) {
    return qg::counters_bytes(num_sms) +
           (size_t)qg::slots_of(num_sms) * qg::ROWS * (size_t)(kv->d + 2) * sizeof(float);
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
    p.unit = (uint32_t)c->unit;
    p.page = (uint32_t)(c->st[1] / c->unit);
    p.head = (uint32_t)(c->st[2] / c->unit);
    p.token = (uint32_t)(c->st[3] / c->unit);
    const bool e4m3 = c->dtype == QGEMM_E4M3;
    if (e4m3) {
        p.ks = c->ks + a.layer * c->sst[0];
        p.vs = c->vs + a.layer * c->sst[0];
        p.sextent = c->sextent - a.layer * c->sst[0];
        p.sunit = (uint32_t)c->sunit;
        p.spage = (uint32_t)(c->sst[1] / c->sunit);
        p.shead = (uint32_t)(c->sst[2] / c->sunit);
        p.stoken = (uint32_t)(c->sst[3] / c->sunit);
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
    p.slots = qg::slots_of(ctx.num_sms);
    p.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + qg::counters_bytes(ctx.num_sms));
    p.err = ctx.err;
    p.one_page = c->page_size % qg::STEP == 0;
    kvi::page_divisor(p.page_size, &p.page_magic, &p.page_shift);
    // no more CTAs than tiles (and EXTRAs) the table rows can hold
    const int64_t most = units * (kvi::tiles_of(a.max_pages * (int32_t)c->page_size, qg::TILE) + 3);
    if (a.bf16)
        return c->d == 64 ? qg::launch_cache<qg::TypeBF16, 64>(p, e4m3, most, ctx)
                          : qg::launch_cache<qg::TypeBF16, 128>(p, e4m3, most, ctx);
    return c->d == 64 ? qg::launch_cache<qg::TypeF16, 64>(p, e4m3, most, ctx)
                      : qg::launch_cache<qg::TypeF16, 128>(p, e4m3, most, ctx);
}

}  // namespace qgi

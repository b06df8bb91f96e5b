// rope_append.cu -- rotary positions, alone or on the way into the paged key-value cache.
//
// A pair (a, b) of a head at position p becomes (a cos t - b sin t, a sin t + b cos t) times the
// magnitude factor, t = p w_i.  The inverse (the rotation's transpose, which is its gradient)
// turns by -t.  Pairs are (2i, 2i + 1) (interleaved) or (i, i + rot_dim / 2) (halves); elements
// past rot_dim pass through.
//
// Angles.  w_i / 2 pi is held as a 64-bit fraction of a turn, so position times frequency modulo
// one turn is one wrapping integer product and adds no error.  The fraction comes from doubles: for w_i of
// at most a radian it is off by less than 2^-53 of a turn (pair 0 of base 10^4: 2^-56.5), so the angle at position p
// by 2^-53 p, 2^-22 of a turn at 2^31 (an fp32 angle at position 10^5 is off by 2^-8 rad).  The top 32 bits are a signed fraction: its leading 24
// go to sincospif, the rest turns the result, so sine and cosine are off by sincospif's error alone.
//
// Appending stores keys (rotated) and values as they are or as E4M3 codes with one power of two
// per 32 elements: X = floor(log2 amax) - 8, code = e4m3_rn(x 2^-X) saturated at 448, straight
// from the fp32 rotation (one rounding).  fp16 sources stop at X = -15: below that 2^-24, the
// half's own quantum, is finer than E4M3's grid, and every code times its scale stays a half.
//
// Bound: memory (one read and one write of every element; at 16384 x 48 rows of 128 about 0.4 GB).
// A block takes the rows (token, head) of a few tokens: the sines and cosines of its tokens are
// computed once into shared memory, while the first rows' loads are already in flight, and the next
// rows' loads are in flight while a row is turned.  Aligned rows go through rope_pair_kernel; the general
// kernel reads 16 bytes a lane, LPR lanes a row, or single elements where rows are not aligned, and takes a
// pair's other half from the lane that holds it (a shuffle) or turns the row in shared memory.
#include "kv_common.cuh"

namespace qg {
namespace {

constexpr int THREADS = 128;
constexpr int BLOCKS = 6;        // resident on an SM (80 registers a thread)
// Of the paired kernel: 72 registers, of which rotation alone at d other than 128 and 16-bit appends as halves spill 8 to
// 20 bytes; 6 blocks spill none.  7 / 6 blocks: 30011 x 12 x 96, rot 48 24.7 / 24.9 us, interleaved rot 38 23.0 / 24.2; 8192 x
// 40 x 96, rot 96 23.8 / 22.4; appends of 16384 x 48 x 128 61.8 / 63.6, of 15009 x 36 x 64 25.1 / 26.5.
constexpr int PAIR_BLOCKS = 7;
constexpr int ROWS = 4;          // rows a lane has in flight
constexpr int HALF_ROWS = 2;     // of half-rotated rows
constexpr int PAIR_ROWS = 2;     // and in the paired kernel, of two pieces each
constexpr int MAX_TPC = 16;      // tokens of one block

struct RopeParams {
    const uint8_t *x[3];         // q, k, v
    int64_t xt[3], xh[3];        // token and head strides, bytes
    uint8_t *y;                  // rotated q
    int64_t yt, yh;
    uint8_t *pk[2], *ps[2];      // cache planes of this layer: data and scales of keys, values
    int64_t page, head, token, spage, shead, stoken;
    int64_t extent, sextent;     // bytes of a plane from this layer's base (debug checks)
    const int32_t *seqs, *pos, *table;
    int64_t table_stride;
    int32_t T, d, hq, hkv, tpc, hsplit;
    int32_t max_seqs, max_pages, page_size, pages;
    int32_t rot;                 // 0: no rotation
    int32_t min_exp;             // smallest X of an E4M3 block
    float mscale, sign;
    int32_t xt32[3], xh32[3], yt32, yh32, head32, shead32;   // the strides, where they fit (paired kernel)
    unsigned *err;
};
struct Frequencies {
    uint64_t f[128];
};

// Floats of a token's cosines, and of its sines.
__host__ __device__ constexpr int table_pitch(int rot) {
    return (rot / 2 + 3) & ~3;
}

// 8 elements of a row from element e0 on; those at d and beyond read as zero.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint8_t *row, int e0, int d) {
    if (e0 >= d) return make_uint4(0, 0, 0, 0);
    if (VEC) return *reinterpret_cast<const uint4 *>(row + 2 * e0);
    uint32_t w[4] = {0, 0, 0, 0};
    const uint16_t *p = reinterpret_cast<const uint16_t *>(row);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (e0 + i < d) w[i / 2] |= uint32_t(p[e0 + i]) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t *row, int e0, int d, uint4 v) {
    if (e0 >= d) return;
    if (VEC) {
        *reinterpret_cast<uint4 *>(row + 2 * e0) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint16_t *p = reinterpret_cast<uint16_t *>(row);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (e0 + i < d) p[e0 + i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
}

// The block's 8 values as E4M3 with the scale of their 32 (four lanes hold a block).  Returns the
// codes; *byte is the UE8M0 scale.  fmaxf passes over NaN, whose code is E4M3's NaN.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], int min_exp, uint32_t *byte) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    // floor(log2) is the exponent field; fp32 subnormals (field 0) are below every X that is kept
    int X = int(__float_as_uint(amax) >> 23) - 127 - 8;
    X = amax > 0.0f ? max(X, min_exp) : 0;
    *byte = uint32_t(X + 127);
    const float inv = __uint_as_float(uint32_t(127 - X) << 23);    // 2^-X, X in [-127, 120]
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
            : "=h"(lo)
            : "f"(x[4 * i + 1] * inv), "f"(x[4 * i] * inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
            : "=h"(hi)
            : "f"(x[4 * i + 3] * inv), "f"(x[4 * i + 2] * inv));
        w[i] = uint32_t(lo) | (uint32_t(hi) << 16);
    }
    return make_uint2(w[0], w[1]);
}

// The slots of the block's tokens in the cache, and their sines and cosines ([token][2][pitch]).
template <bool CACHE>
__device__ __forceinline__ void set_up(const RopeParams &p, const Frequencies &fr, int t0, int nt, int pitch,
                                       float *s_cs, int64_t *s_slot, int64_t *s_sslot) {
    const int tid = threadIdx.x, half = p.rot / 2;
    if (CACHE && tid < nt) {
        const int t = t0 + tid, seq = p.seqs[t];
        int32_t page = 0, off = 0;
        bool ok = seq >= 0 && seq < p.max_seqs;
        ok = ok && kvi::locate(p.table + seq * p.table_stride, p.max_pages, p.page_size, p.pages,
                               p.pos[t], &page, &off);
        if (!ok) report_index(p.err);
        s_slot[tid] = ok ? page * p.page + off * p.token : -1;
        s_sslot[tid] = page * p.spage + off * p.stoken;
    }
    for (int i = tid; i < nt * half; i += THREADS) {
        const int t = i / half, j = i - t * half;
        const uint64_t turn = uint64_t(int64_t(p.pos[t0 + t])) * fr.f[j];
        // the top 32 bits as a signed fraction of half a turn: the 24 an fp32 holds, and the angle of
        // the rest, which turns the result by the first two terms of its series
        const int32_t top = int32_t(turn >> 32);
        const float x = float(top);
        const float rest = float(top - (x < 0x1p31f ? int32_t(x) : 0x7FFFFFFF)) * (3.14159265358979f * 0x1p-31f);
        float s, c;
        sincospif(x * 0x1p-31f, &s, &c);
        s_cs[(2 * t) * pitch + j] = (c - rest * s) * p.mscale;
        s_cs[(2 * t + 1) * pitch + j] = (s + rest * c) * (p.mscale * p.sign);
    }
}

// LPR lanes a row of 8 elements each; INTER: interleaved pairs; VEC: rows are 16-byte aligned and d a
// multiple of 8; CACHE: 0 none (rotation alone), 1 planes of the activations' type, 2 E4M3.  Halves whose
// length is a multiple of 8 take a pair's other piece from the lane that holds it; of any other length it lies
// across two lanes' pieces, so a row's lanes lay the row into shared memory, turn a pair each and take their
// turned elements from there in 32 bits.  (30011 x 12 rows of 96, rot 38: 39.9 us; the two pieces read and
// shifted 47.4; every element's other half from memory 93.6.  8192 x 40 rows of 120, rot 96: 33.4 us, by shared memory
// 39.8.)
template <class TY, int LPR, bool INTER, bool VEC, int CACHE>
__global__ void __launch_bounds__(THREADS, BLOCKS) rope_append_kernel(const __grid_constant__ RopeParams p,
                                                              const __grid_constant__ Frequencies fr) {
    extern __shared__ __align__(16) float s_cs[];      // [tpc][2][pitch]: cosines, sines
    __shared__ int64_t s_slot[MAX_TPC], s_sslot[MAX_TPC];
    constexpr int NR = INTER ? ROWS : HALF_ROWS;
    // halves: rows as read and as turned; an eighth more a row, so that a warp's rows lie in different banks
    constexpr int XP = 9 * LPR / 8, YP = 9 * LPR;      // of 16 bytes; of floats
    __shared__ uint4 s_x[INTER ? 1 : NR * (THREADS / LPR) * XP];
    __shared__ __align__(16) float s_y[INTER ? 1 : NR * (THREADS / LPR) * YP];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, half = p.rot / 2, pitch = table_pitch(p.rot);
    const int t0 = blockIdx.x * p.tpc, nt = min(p.tpc, p.T - t0);
    constexpr int RPP = THREADS / LPR;                 // rows a pass
    const int lane_r = tid % LPR;
    const int e0 = 8 * lane_r;
    const int heads = p.hq + (CACHE ? 2 * p.hkv : 0);
    // this block's heads (few tokens: a token's heads are dealt to several blocks)
    const int h0 = heads * int(blockIdx.y) / p.hsplit, nh = heads * int(blockIdx.y + 1) / p.hsplit - h0;

    // This lane's rows, RPP apart in the order token, head: the next one without a division.
    struct Row {
        int t, h;
    };
    const int dt = RPP / nh, dh = RPP - dt * nh;
    auto next = [&](Row &r) {
        r.t += dt;
        r.h += dh;
        if (r.h >= nh) {
            r.h -= nh;
            ++r.t;
        }
    };
    // Which of q, k, v the row is of, and its head there.
    auto side_of = [&](const Row &r, int &h) {
        h = h0 + r.h;
        if (!CACHE || h < p.hq) return 0;
        h -= p.hq;
        if (h < p.hkv) return 1;
        h -= p.hkv;
        return 2;
    };
    auto source = [&](const Row &r) {
        int h;
        const int side = side_of(r, h);
        const uint8_t *x = side == 0 ? p.x[0] : (side == 1 ? p.x[1] : p.x[2]);
        const int64_t xt = side == 0 ? p.xt[0] : (side == 1 ? p.xt[1] : p.xt[2]);
        const int64_t xh = side == 0 ? p.xh[0] : (side == 1 ? p.xh[1] : p.xh[2]);
        return x + (t0 + r.t) * xt + h * xh;
    };
    auto fetch = [&](Row r, uint4 (&v)[NR]) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if (r.t < nt) v[i] = load8<VEC>(source(r), e0, p.d);
            next(r);
        }
        return r;
    };
    const int r0 = tid / LPR;
    Row row = {r0 / nh, r0 % nh};
    uint4 v[NR];
    Row ahead = fetch(row, v);

    set_up<CACHE != 0>(p, fr, t0, nt, pitch, s_cs, s_slot, s_sslot);
    __syncthreads();

    const bool whole = half % 8 == 0;                  // pieces' partners are pieces

    // every lane of the block makes the same number of rounds (the rows' exchanges are by warp)
    for (int done = 0; done < nt * nh; done += NR * RPP) {
        // the next rows' loads are in flight while these are turned: an output that is the input
        // itself is read before it is written, rows never share elements
        uint4 w[NR];
        const Row after = fetch(ahead, w);
        if (!INTER && half > 0 && !whole) {
            __syncwarp();                               // the last round's rows have been read
#pragma unroll
            for (int i = 0; i < NR; ++i) s_x[(i * RPP + r0) * XP + lane_r] = v[i];
            __syncwarp();
            Row r = row;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                int h;
                if (r.t < nt && side_of(r, h) < 2) {
                    const uint16_t *x = reinterpret_cast<const uint16_t *>(s_x + (i * RPP + r0) * XP);
                    float *y = s_y + (i * RPP + r0) * YP;
                    const float *cs = s_cs + (2 * r.t) * pitch, *sn = cs + pitch;
                    for (int j = lane_r; j < half; j += LPR) {
                        const float a = TY::unpack(x[j]).x, b = TY::unpack(x[j + half]).x, c = cs[j], s = sn[j];
                        y[j] = a * c - b * s;
                        y[j + half] = a * s + b * c;
                    }
                }
                next(r);
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if (done + i * RPP >= nt * nh) break;       // the same for every lane
            const bool live = row.t < nt;
            const int t = live ? row.t : 0;
            int h;
            const int side = side_of(row, h);
            float x[8];
            {
                const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = TY::unpack(u[j]);
                    x[2 * j] = f.x;
                    x[2 * j + 1] = f.y;
                }
            }
            const bool turned = live && half > 0 && (!CACHE || side < 2);
            const float *cs = s_cs + (2 * t) * pitch, *sn = cs + pitch;
            if (INTER) {
                if (turned && e0 < p.rot) {
                    const float4 c = *reinterpret_cast<const float4 *>(cs + e0 / 2);
                    const float4 s = *reinterpret_cast<const float4 *>(sn + e0 / 2);
                    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (e0 / 2 + j < half) {
                            const float a = x[2 * j], b = x[2 * j + 1];
                            x[2 * j] = a * cc[j] - b * ss[j];
                            x[2 * j + 1] = a * ss[j] + b * cc[j];
                        }
                }
            } else if (whole) {
                // the other halves of this lane's pairs are in the lane half / 8 further or back
                const int hl = half / 8;
                const bool first = lane_r < hl, in = lane_r < 2 * hl;
                const int other = in ? (tid & 31) + (first ? hl : -hl) : 0;
                const uint32_t flip = first ? 0x80008000u : 0u;     // the sine's sign, on both
                const uint32_t ow[4] = {__shfl_sync(0xFFFFFFFFu, v[i].x, other) ^ flip,
                                        __shfl_sync(0xFFFFFFFFu, v[i].y, other) ^ flip,
                                        __shfl_sync(0xFFFFFFFFu, v[i].z, other) ^ flip,
                                        __shfl_sync(0xFFFFFFFFu, v[i].w, other) ^ flip};
                if (turned && in) {
                    const int j0 = first ? e0 : e0 - half;
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const float4 c = *reinterpret_cast<const float4 *>(cs + j0 + j);
                        const float4 s = *reinterpret_cast<const float4 *>(sn + j0 + j);
                        const float2 o0 = TY::unpack(ow[j / 2]), o1 = TY::unpack(ow[j / 2 + 1]);
                        const float o[4] = {o0.x, o0.y, o1.x, o1.y};
                        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[j + k] = x[j + k] * cc[k] + o[k] * ss[k];
                    }
                }
            } else if (turned && e0 < p.rot) {
                const float *y = s_y + (i * RPP + r0) * YP + e0;
                const float4 lo = *reinterpret_cast<const float4 *>(y), hi = *reinterpret_cast<const float4 *>(y + 4);
                const float yy[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (e0 + j < p.rot) x[j] = yy[j];
            }
            uint32_t byte = 0;
            uint2 codes = make_uint2(0, 0);
            // every lane of a warp that has a key or a value: it shuffles
            if (CACHE == 2 && __any_sync(0xFFFFFFFFu, live && side > 0))
                codes = quantise8(x, p.min_exp, &byte);
            const uint4 out = make_uint4(TY::pack(x[0], x[1]), TY::pack(x[2], x[3]),
                                         TY::pack(x[4], x[5]), TY::pack(x[6], x[7]));
            if (live) {
                if (side == 0) {
                    store8<VEC>(p.y + (t0 + t) * p.yt + h * p.yh, e0, p.d, out);
                } else if (s_slot[t] >= 0 && e0 < p.d) {
                    const int64_t at = s_slot[t] + h * p.head;
                    uint8_t *plane = side == 1 ? p.pk[0] : p.pk[1];
                    if (CACHE == 2) {
                        const int64_t sat = s_sslot[t] + h * p.shead;
                        if (QG_IN_BOUNDS(p.err, at >= 0 && at + p.d <= p.extent &&
                                                    sat >= 0 && sat + p.d / 32 <= p.sextent)) {
                            *reinterpret_cast<uint2 *>(plane + at + e0) = codes;
                            if (lane_r % 4 == 0)
                                (side == 1 ? p.ps[0] : p.ps[1])[sat + lane_r / 4] = static_cast<uint8_t>(byte);
                        }
                    } else if (QG_IN_BOUNDS(p.err, at >= 0 && at + 2 * p.d <= p.extent)) {
                        *reinterpret_cast<uint4 *>(plane + at + 2 * e0) = out;   // planes are aligned
                    }
                }
            }
            next(row);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) v[i] = w[i];
        row = ahead;
        ahead = after;
    }
}

// The aligned case: a lane takes 16 elements as two pieces of 8, so that for halves both elements of its
// pairs are its own (no exchange, one sine and cosine for two outputs) and what a row costs besides its
// elements is spent once for 16.  Halves: piece k of the first half and of the second for k < rot / 16, then
// the two halves of what is not rotated; interleaved: piece k of the row's first half and of its second.
// Needs rows 16-byte aligned, strides below 2^31 bytes, d a multiple of 16, for halves
// rot of 16, and for E4M3, whose blocks of 32 are four neighbouring lanes' pieces, of 64.  LPR = d / 16 lanes a row (a
// cache's d is 64 or 128), or 0 for lanes counted from d: rotation alone, where no lane needs another, at d = 128
// one percent slower.  Elsewhere the kernel above, 8 elements a lane, bound by its instructions.  (30011 x 12 rows
// of 96, rot 48, fp16: 24.6 us, 5.6 TB/s, against 32.8; interleaved, rot 38: 23.0 against 29.8; 15009 x 36 rows of 128 into
// E4M3: 43.6, 6.0 TB/s, against 62.4; 16384 x 48 rows of 128 into bf16: 61.1, 6.6 TB/s, against 70.6; 8192 x 40
// interleaved rows of 128, bf16: 26.7, 6.3 TB/s, against 28.3.)
template <class TY, int LPR, bool INTER, int CACHE>
__global__ void __launch_bounds__(THREADS, PAIR_BLOCKS) rope_pair_kernel(const __grid_constant__ RopeParams p,
                                                            const __grid_constant__ Frequencies fr) {
    griddep_launch_dependents();
    griddep_wait();
    extern __shared__ __align__(16) float s_cs[];
    __shared__ int64_t s_slot[MAX_TPC], s_sslot[MAX_TPC];
    const int tid = threadIdx.x, half = p.rot / 2, pitch = table_pitch(p.rot);
    const int t0 = blockIdx.x * p.tpc, nt = min(p.tpc, p.T - t0);
    const int lpr = LPR ? LPR : p.d / 16, RPP = THREADS / lpr;
    constexpr int PR = PAIR_ROWS;
    const int r0 = tid / lpr, k = tid - r0 * lpr;
    const bool lane = r0 < RPP;                        // the last lanes may make no whole row
    const int heads = p.hq + (CACHE ? 2 * p.hkv : 0);
    const int h0 = heads * int(blockIdx.y) / p.hsplit, nh = heads * int(blockIdx.y + 1) / p.hsplit - h0;

    // the lane's two pieces, and whether they are rotated
    int ea, eb;
    bool turn_a, turn_b;
    if (INTER) {
        ea = 8 * k;
        eb = p.d / 2 + 8 * k;
        turn_a = ea < p.rot;
        turn_b = eb < p.rot;
    } else {
        const int hl = p.rot / 16, rest = (p.d - p.rot) / 16;
        turn_a = turn_b = k < hl;
        ea = turn_a ? 8 * k : p.rot + 8 * (k - hl);
        eb = turn_a ? half + 8 * k : p.rot + 8 * (rest + k - hl);
    }
    turn_a = turn_a && lane;
    turn_b = turn_b && lane;

    struct Row {
        int t, h;
    };
    const int dt = RPP / nh, dh = RPP - dt * nh;
    auto next = [&](Row &r) {
        r.t += dt;
        r.h += dh;
        if (r.h >= nh) {
            r.h -= nh;
            ++r.t;
        }
    };
    auto side_of = [&](const Row &r, int &h) {
        h = h0 + r.h;
        if (!CACHE || h < p.hq) return 0;
        h -= p.hq;
        if (h < p.hkv) return 1;
        h -= p.hkv;
        return 2;
    };
    auto fetch = [&](Row r, uint4 (&a)[PR], uint4 (&b)[PR]) {
#pragma unroll
        for (int i = 0; i < PR; ++i) {
            if (r.t < nt && lane) {
                int h;
                const int side = side_of(r, h);
                const uint8_t *x = side == 0 ? p.x[0] : (side == 1 ? p.x[1] : p.x[2]);
                const int32_t xt = side == 0 ? p.xt32[0] : (side == 1 ? p.xt32[1] : p.xt32[2]);
                const int32_t xh = side == 0 ? p.xh32[0] : (side == 1 ? p.xh32[1] : p.xh32[2]);
                const uint8_t *row = x + int64_t(t0 + r.t) * xt + int64_t(h) * xh;
                a[i] = *reinterpret_cast<const uint4 *>(row + 2 * ea);
                b[i] = *reinterpret_cast<const uint4 *>(row + 2 * eb);
            }
            next(r);
        }
        return r;
    };
    auto unpack = [](const uint4 &v, float (&x)[8]) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = TY::unpack(u[j]);
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
        }
    };
    auto pack = [](const float (&x)[8]) {
        return make_uint4(TY::pack(x[0], x[1]), TY::pack(x[2], x[3]), TY::pack(x[4], x[5]), TY::pack(x[6], x[7]));
    };
    auto pairs = [&](float (&x)[8], int e, const float *cs, const float *sn) {     // interleaved pairs of a piece
        const float4 c = *reinterpret_cast<const float4 *>(cs + e / 2), s = *reinterpret_cast<const float4 *>(sn + e / 2);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (e / 2 + j >= half) continue;
            const float u = x[2 * j], v = x[2 * j + 1];
            x[2 * j] = u * cc[j] - v * ss[j];
            x[2 * j + 1] = u * ss[j] + v * cc[j];
        }
    };

    Row row = {r0 / nh, r0 % nh};
    uint4 va[PR], vb[PR];
    Row ahead = fetch(row, va, vb);
    set_up<CACHE != 0>(p, fr, t0, nt, pitch, s_cs, s_slot, s_sslot);
    __syncthreads();

    for (int done = 0; done < nt * nh; done += PR * RPP) {
        uint4 wa[PR], wb[PR];
        const Row after = fetch(ahead, wa, wb);        // in flight while these are turned
#pragma unroll
        for (int i = 0; i < PR; ++i) {
            const bool live = row.t < nt && lane;
            const int t = row.t < nt ? row.t : 0;
            int h;
            const int side = side_of(row, h);
            next(row);
            float a[8], b[8];
            unpack(va[i], a);
            unpack(vb[i], b);
            const bool rotate = p.rot > 0 && (!CACHE || side < 2);
            const float *cs = s_cs + (2 * t) * pitch, *sn = cs + pitch;
            if (INTER) {
                if (rotate && turn_a) pairs(a, ea, cs, sn);
                if (rotate && turn_b) pairs(b, eb, cs, sn);
            } else if (rotate && turn_a) {
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const float4 c = *reinterpret_cast<const float4 *>(cs + ea + j);
                    const float4 s = *reinterpret_cast<const float4 *>(sn + ea + j);
                    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float u = a[j + q], v = b[j + q];
                        a[j + q] = u * cc[q] - v * ss[q];
                        b[j + q] = u * ss[q] + v * cc[q];
                    }
                }
            }
            if (!CACHE || side == 0) {
                if (live) {
                    uint8_t *y = p.y + int64_t(t0 + t) * p.yt32 + int64_t(h) * p.yh32;
                    *reinterpret_cast<uint4 *>(y + 2 * ea) = pack(a);
                    *reinterpret_cast<uint4 *>(y + 2 * eb) = pack(b);
                }
            }
            if (CACHE == 2) {
                // every lane of a warp that has a key or a value: it shuffles
                if (__any_sync(0xFFFFFFFFu, live && side > 0)) {
                    uint32_t ba, bb;
                    const uint2 ca = quantise8(a, p.min_exp, &ba), cb = quantise8(b, p.min_exp, &bb);
                    if (live && side > 0 && s_slot[t] >= 0) {
                        const int64_t at = s_slot[t] + int64_t(h) * p.head32, sat = s_sslot[t] + int64_t(h) * p.shead32;
                        if (QG_IN_BOUNDS(p.err, at >= 0 && at + p.d <= p.extent && sat >= 0 &&
                                                    sat + p.d / 32 <= p.sextent)) {
                            uint8_t *plane = (side == 1 ? p.pk[0] : p.pk[1]) + at;
                            *reinterpret_cast<uint2 *>(plane + ea) = ca;
                            *reinterpret_cast<uint2 *>(plane + eb) = cb;
                            if (k % 4 == 0) {
                                uint8_t *scales = (side == 1 ? p.ps[0] : p.ps[1]) + sat;
                                scales[ea / 32] = static_cast<uint8_t>(ba);
                                scales[eb / 32] = static_cast<uint8_t>(bb);
                            }
                        }
                    }
                }
            } else if (CACHE == 1 && live && side > 0 && s_slot[t] >= 0) {
                const int64_t at = s_slot[t] + int64_t(h) * p.head32;
                if (QG_IN_BOUNDS(p.err, at >= 0 && at + 2 * p.d <= p.extent)) {
                    uint8_t *plane = (side == 1 ? p.pk[0] : p.pk[1]) + at;
                    *reinterpret_cast<uint4 *>(plane + 2 * ea) = pack(a);
                    *reinterpret_cast<uint4 *>(plane + 2 * eb) = pack(b);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < PR; ++i) {
            va[i] = wa[i];
            vb[i] = wb[i];
        }
        row = ahead;
        ahead = after;
    }
}

template <class TY, int LPR, int CACHE>
cudaError_t launch_pair(const RopeParams &p, const Frequencies &fr, bool inter, dim3 grid, size_t smem,
                        cudaStream_t stream) {
    return inter ? launch_dependent(rope_pair_kernel<TY, LPR, true, CACHE>, grid, THREADS, smem, stream, p, fr)
                 : launch_dependent(rope_pair_kernel<TY, LPR, false, CACHE>, grid, THREADS, smem, stream, p, fr);
}

template <class TY>
cudaError_t launch_pair_type(const RopeParams &p, const Frequencies &fr, bool inter, int cache, dim3 grid, size_t smem,
                             cudaStream_t stream) {
    if (cache == 2)
        return p.d <= 64 ? launch_pair<TY, 4, 2>(p, fr, inter, grid, smem, stream)
                         : launch_pair<TY, 8, 2>(p, fr, inter, grid, smem, stream);
    if (cache == 1)
        return p.d <= 64 ? launch_pair<TY, 4, 1>(p, fr, inter, grid, smem, stream)
                         : launch_pair<TY, 8, 1>(p, fr, inter, grid, smem, stream);
    if (p.d == 128) return launch_pair<TY, 8, 0>(p, fr, inter, grid, smem, stream);
    return launch_pair<TY, 0, 0>(p, fr, inter, grid, smem, stream);
}

template <class TY, int LPR, bool INTER, bool VEC, int CACHE>
cudaError_t launch(const RopeParams &p, const Frequencies &fr, dim3 grid, size_t smem,
                   cudaStream_t stream) {
    return launch_dependent(rope_append_kernel<TY, LPR, INTER, VEC, CACHE>, grid, THREADS, smem, stream, p, fr);
}

template <class TY, int LPR, int CACHE>
cudaError_t launch_layout(const RopeParams &p, const Frequencies &fr, bool inter, bool vec,
                          dim3 grid, size_t smem, cudaStream_t stream) {
    if (inter) return vec ? launch<TY, LPR, true, true, CACHE>(p, fr, grid, smem, stream)
                          : launch<TY, LPR, true, false, CACHE>(p, fr, grid, smem, stream);
    return vec ? launch<TY, LPR, false, true, CACHE>(p, fr, grid, smem, stream)
               : launch<TY, LPR, false, false, CACHE>(p, fr, grid, smem, stream);
}

template <class TY>
cudaError_t launch_type(const RopeParams &p, const Frequencies &fr, bool inter, bool vec, int cache,
                        dim3 grid, size_t smem, cudaStream_t stream) {
    if (cache == 2)      // a cache's d is 64 or 128
        return p.d <= 64 ? launch_layout<TY, 8, 2>(p, fr, inter, vec, grid, smem, stream)
                         : launch_layout<TY, 16, 2>(p, fr, inter, vec, grid, smem, stream);
    if (cache == 1)
        return p.d <= 64 ? launch_layout<TY, 8, 1>(p, fr, inter, vec, grid, smem, stream)
                         : launch_layout<TY, 16, 1>(p, fr, inter, vec, grid, smem, stream);
    if (p.d <= 64) return launch_layout<TY, 8, 0>(p, fr, inter, vec, grid, smem, stream);
    if (p.d <= 128) return launch_layout<TY, 16, 0>(p, fr, inter, vec, grid, smem, stream);
    return launch_layout<TY, 32, 0>(p, fr, inter, vec, grid, smem, stream);
}

}  // namespace
}  // namespace qg

namespace qgi {

cudaError_t launch_rope_append(const AppendArgs &a, const LaunchCtx &ctx) {
    qg::RopeParams p = {};
    qg::Frequencies fr = {};
    const bool append = a.kv != nullptr;
    auto aligned = [](const void *b, int64_t ts, int64_t hs) {
        return reinterpret_cast<uintptr_t>(b) % 16 == 0 && ts % 8 == 0 && hs % 8 == 0;
    };
    bool vec = a.d % 8 == 0;
    p.hq = a.q.heads;
    if (p.hq > 0) {
        p.x[0] = static_cast<const uint8_t *>(a.q.x);
        p.xt[0] = 2 * a.q.xt;
        p.xh[0] = 2 * a.q.xh;
        p.y = static_cast<uint8_t *>(a.q.y);
        p.yt = 2 * a.q.yt;
        p.yh = 2 * a.q.yh;
        vec = vec && aligned(a.q.x, a.q.xt, a.q.xh) && aligned(a.q.y, a.q.yt, a.q.yh);
    }
    bool e4m3 = false;
    if (append) {
        const qgemm_kv_cache *c = a.kv;
        e4m3 = c->dtype == QGEMM_E4M3;
        p.x[1] = static_cast<const uint8_t *>(a.k);
        p.x[2] = static_cast<const uint8_t *>(a.v);
        p.xt[1] = 2 * a.kt;
        p.xh[1] = 2 * a.kh;
        p.xt[2] = 2 * a.vt;
        p.xh[2] = 2 * a.vh;
        vec = vec && aligned(a.k, a.kt, a.kh) && aligned(a.v, a.vt, a.vh);
        p.hkv = (int32_t)c->heads;
        p.pk[0] = c->k + a.layer * c->st[0];
        p.pk[1] = c->v + a.layer * c->st[0];
        p.extent = c->extent - a.layer * c->st[0];
        p.page = c->st[1];
        p.head = c->st[2];
        p.token = c->st[3];
        if (e4m3) {
            p.ps[0] = c->ks + a.layer * c->sst[0];
            p.ps[1] = c->vs + a.layer * c->sst[0];
            p.sextent = c->sextent - a.layer * c->sst[0];
            p.spage = c->sst[1];
            p.shead = c->sst[2];
            p.stoken = c->sst[3];
        }
        p.page_size = (int32_t)c->page_size;
        p.pages = (int32_t)c->pages;
        p.seqs = a.seqs;
        p.table = a.table;
        p.table_stride = a.table_stride;
        p.max_seqs = a.max_seqs;
        p.max_pages = a.max_pages;
    }
    p.pos = a.pos;
    p.T = a.T;
    p.d = a.d;
    p.min_exp = a.bf16 ? -127 : -15;
    p.mscale = 1.0f;
    p.sign = a.inverse ? -1.0f : 1.0f;
    p.err = ctx.err;
    bool inter = true;
    if (a.rope) {
        p.rot = a.rope->rot_dim;
        p.mscale = a.rope->mscale;
        inter = a.rope->interleaved != 0;
        for (int i = 0; i < p.rot / 2; ++i) fr.f[i] = a.rope->freq[i];
    }
    // Tokens a block: at most the rows of three rounds of what its lanes hold, five with an E4M3 cache (whose slots
    // are another chain of reads at a block's start), and in the general kernel four, eight for halves (30011 x 12 rows of
    // 96, rot 38, four / six / eight: 41.2 / 39.8 / 39.9 us; 8192 x 40 of 128, rot 40: 39.5 / 35.8 / 35.3); more leaves the last
    // blocks alone on the GPU, fewer computes the sines for too few rows.  With few tokens one token a
    // block and its heads dealt to several blocks, two blocks an SM.  A row more starts a round for
    // itself: 30011 x 12 rows of 96, 42 a round, 10 tokens 24.6 us and 11 26.1.  (Paired kernel, tokens a block: 8192 x 40
    // rows of 128 1 / 2 / 4 / 8: 31.4 / 26.5 / 27.3 / 29.6 us; 6038 x 26 1 / 3 / 5 / 8: 17.3 / 14.9 / 17.1 / 16.6; 15009 x
    // 36 into E4M3 2 / 4 / 8: 48.3 / 43.5 / 45.8.)
    const int heads = p.hq + 2 * p.hkv;
    bool pair = vec && a.d % 16 == 0 && (inter || p.rot % (e4m3 ? 64 : 16) == 0);
    auto fits = [&](int64_t stride, int32_t *to) {
        pair = pair && stride <= INT32_MAX;
        *to = (int32_t)(pair ? stride : 0);
    };
    for (int i = 0; i < 3; ++i) {
        fits(p.xt[i], &p.xt32[i]);
        fits(p.xh[i], &p.xh32[i]);
    }
    fits(p.yt, &p.yt32);
    fits(p.yh, &p.yh32);
    fits(p.head, &p.head32);
    fits(p.shead, &p.shead32);
    int lpr = a.d <= 64 ? 8 : (a.d <= 128 ? 16 : 32);
    if (pair) lpr = a.d / 16;
    const int rpp = qg::THREADS / lpr;
    const int64_t slots = 2 * (int64_t)ctx.num_sms;
    const int rows = pair ? (e4m3 ? 5 : 3) * qg::PAIR_ROWS * rpp : 4 * qg::ROWS * rpp;
    int tpc = rows / heads;
    if (tpc < 1) tpc = 1;
    if (tpc > qg::MAX_TPC) tpc = qg::MAX_TPC;
    while (tpc > 1 && ((int64_t)a.T + tpc - 1) / tpc < slots) --tpc;
    p.tpc = tpc;
    int64_t split = a.T < slots ? slots / a.T : 1;
    const int64_t most = (heads + rpp - 1) / rpp;
    p.hsplit = (int32_t)(split < most ? split : most);
    const dim3 grid((unsigned)((a.T + tpc - 1) / tpc), (unsigned)p.hsplit);
    const size_t smem = sizeof(float) * (size_t)tpc * 2 * qg::table_pitch(p.rot);
    const int cache = append ? (e4m3 ? 2 : 1) : 0;
    if (pair)
        return a.bf16 ? qg::launch_pair_type<qg::TypeBF16>(p, fr, inter, cache, grid, smem, ctx.stream)
                      : qg::launch_pair_type<qg::TypeF16>(p, fr, inter, cache, grid, smem, ctx.stream);
    return a.bf16 ? qg::launch_type<qg::TypeBF16>(p, fr, inter, vec, cache, grid, smem, ctx.stream)
                  : qg::launch_type<qg::TypeF16>(p, fr, inter, vec, cache, grid, smem, ctx.stream);
}

}  // namespace qgi

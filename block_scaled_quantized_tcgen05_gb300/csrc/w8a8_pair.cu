// w8a8_pair.cu -- product of 8-bit integers on CTA pairs, both operands as halves on the fp16 tensor cores.
//
//   C[m, n] = round( (sum_k A[m, k] W[n, k]) * sa[m] * sw[n] [+ bias[n]] [+ C_old] ), then ReLU.
//
// sm_103a has no integer tensor core worth the name (mma.sync on s8 runs at the rate of dp4a, 251 products a
// clock and SM against about 4096 on tcgen05 kind::f16; measured), and every int8 is a half, whose products are
// exact in the fp32 accumulator as long as the sum stays below 2^24.  So the product D[n, m] = sum_k W[n, k]
// A[m, k] runs on kind::f16:
//
//   * weights are the left operand: raw bytes land in shared memory by TMA (64 a row, 64-byte swizzle), converter
//     warps turn them into halves in registers and write them to TMEM, from where the MMA reads them.  They never
//     take shared memory's bandwidth as halves;
//   * tokens are the right operand, in shared memory.  They are turned into halves once, by a kernel ahead of this
//     one into pooled scratch, because every block of weight rows reads them again;
//   * a cluster of two CTAs computes 256 weight rows x BT tokens, each CTA holding 128 weight rows in TMEM and BT / 2 tokens
//     in shared memory;
//   * the epilogue reads D (lane = weight row, column = token), applies the scales, and writes through shared
//     memory and TMA stores where C allows a tensor map;
//   * tiles go to the pairs in whole waves; what is left after them (all, where there are fewer tiles than pairs) is
//     cut into equal ranges of K, one a pair, whatever tiles they cover: a tile that several pairs share leaves fp32 partial
//     sums in scratch, which a reduction kernel adds in the order of K.  (The warp that finishes a piece last adding them at the
//     kernel's end instead: 4096 x 14336 x 4096 in 310 us against 294, 256 x 4096 x 4096 29 against 21: too few loads in flight.)
//
// Measured: 8192^3 543 - 566 us (1.94 - 2.02 PFLOP/s, what the library's bf16 product reaches), 4096 x 14336 x 4096 246 us, 4096^3 83 (issued
// one after another for long, under the power cap, 580 - 590 and 261 - 264);
// 64 x 28672 x 8192 44 us (5.4 TB/s of weights; 6.3 in the middle, the rest start and end), 333 x 5003 x 4111 19 us: the tokens' halves 4, the k-tiles 11, epilogue, partial sums and launches the rest.
#include <algorithm>
#include <type_traits>

#include "qgemm_common.cuh"
#include "w8a8_common.cuh"

namespace {

using namespace qg;

constexpr int BW = 128;                 // weight rows per CTA (256 per pair: the MMA's M)
constexpr int EPI_WARPS = 8;            // two per lane quarter, one per half of the tokens
constexpr int CONV_WARP0 = 2 + EPI_WARPS;
constexpr int CONV_WARPS = 8;           // two per lane quarter: alternate stages of 64 k, or a half each of every 128 k
constexpr int THREADS = 32 * (CONV_WARP0 + CONV_WARPS + 1);
constexpr uint32_t TMEM_COLS = 512;

template <int BT>
struct Cfg {
    static constexpr int BK = BT == 256 ? 64 : 128;                           // k per stage
    static constexpr int STAGES = BT == 256 ? 6 : BT == 128 ? 4 : 6;          // tokens' tiles and the weights' slots in TMEM
    static constexpr int RAWS = BT == 256 ? 6 : BT == 128 ? 7 : 8;            // raw weights' tiles: their slots are free once converted
    static constexpr int BUFS = BT == 256 ? 1 : 2;                            // accumulators: the next tile's MMAs beside the epilogue
    static constexpr int WPROD_WARP = CONV_WARP0 + CONV_WARPS;
    static constexpr int TURNS = BK == 64 ? 2 : 1;                            // a converter warp takes every TURNS-th stage
    // A warp that passes over stages must come back to the same ones: it would otherwise miss phases of their barriers, whose
    // parity then no longer tells them apart.
    static_assert(STAGES % TURNS == 0 && RAWS % TURNS == 0, "stages in turn");
    static constexpr uint32_t A_COLS = BK / 2;                                // TMEM columns of a stage's weights
    static constexpr uint32_t X_HALF = (BT / 2) * 128;                        // 64 k of the tokens: rows of 128 bytes
    static constexpr uint32_t X_BYTES = X_HALF * (BK / 64);
    static constexpr uint32_t RAW_BYTES = BW * BK;
    static constexpr uint32_t STAGE_TX = 2 * X_BYTES;                         // both CTAs' tokens, on the leader
    static constexpr int CHUNKS = BT / 64;                                    // 32-token chunks of an epilogue warp
    static constexpr uint32_t EPI_BYTES = CHUNKS * 2048;
    static constexpr uint32_t OFF_RAW = STAGES * X_BYTES;
    static constexpr uint32_t OFF_EPI = OFF_RAW + RAWS * RAW_BYTES;
    static constexpr uint32_t OFF_SA = OFF_EPI + EPI_WARPS * EPI_BYTES;       // each epilogue warp's token scales
    static constexpr uint32_t OFF_BAR = OFF_SA + EPI_WARPS * (BT / 2) * 4;
    static constexpr uint32_t OFF_SLOT = OFF_BAR + (2 * STAGES + 2 * RAWS + 2 * BUFS + 1) * 8;
    static constexpr uint32_t SMEM = OFF_SLOT + 16 + 1024;
    static constexpr uint32_t A_COL0 = BUFS * BT;                             // after the accumulators
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(A_COL0 + STAGES * A_COLS <= TMEM_COLS, "TMEM budget");
    // kind::f16: D fp32, A and B fp16, K-major, N = BT tokens, M = 256 weight rows (pair)
    static constexpr uint32_t IDESC = (1u << 4) | (uint32_t(BT >> 3) << 17) | (uint32_t(256 >> 4) << 24);
};

// Two sums of a column: (sum * sa) * sw + bias.
__device__ __forceinline__ void scaled2(float &x0, float &x1, float s0, float s1, float sa0, float sa1, float sw, float bias) {
    float t0, t1;
    fma2(t0, t1, s0, s1, sa0, sa1, -0.0f, -0.0f);                  // the product itself: x + -0 is x
    fma2(x0, x1, t0, t1, sw, sw, bias, bias);
}

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// The pairs' work: `full` tiles in whole waves over `pairs` pairs, then the other `rest` tiles: one a pair (sharers ==
// rest), or their k-tiles (units) in equal ranges over more sharers, none of them empty (rest < sharers <= pairs).  Units times
// sharers stay below 2^31, so ranges are found in 32 bits.
struct Shares {
    int pairs, full, rest, sharers, KT;
    __host__ __device__ bool shared() const { return sharers > rest; }
    __device__ uint32_t begin(uint32_t p) const { return p * rest * KT / sharers; }
    // the pair whose range holds unit u: the last p with p units / sharers < u + 1
    __device__ uint32_t owner(uint32_t u) const { return ((u + 1) * sharers - 1) / (uint32_t(rest) * KT); }
};

// The items of one pair in order: (tile, k-tiles kt0 .. kt1, slot of its partial sums or -1 for a whole tile).
struct Items {
    const Shares &s;
    int p, i;
    uint32_t u0, u, u1;
    __device__ Items(const Shares &sh, int pair) : s(sh), p(pair), i(pair), u0(0), u(0), u1(0) {
        if (pair >= sh.sharers) return;
        if (sh.shared()) {
            u0 = u = sh.begin(pair);
            u1 = sh.begin(pair + 1);
        } else {
            u1 = 1;                              // its one tile
        }
    }
    __device__ __forceinline__ bool next(int &tile, int &kt0, int &kt1, int &slot) {
        slot = -1;
        kt0 = 0;
        kt1 = s.KT;
        if (i < s.full) {
            tile = i;
            i += s.pairs;
            return true;
        }
        if (u >= u1) return false;
        if (!s.shared()) {
            tile = s.full + p;
            u = u1;
            return true;
        }
        const uint32_t t = u / s.KT;
        tile = s.full + static_cast<int>(t);
        kt0 = static_cast<int>(u - t * s.KT);
        kt1 = min(s.KT, kt0 + static_cast<int>(u1 - u));
        if (kt1 - kt0 < s.KT) slot = 2 * p + (u == u0 ? 0 : 1);
        u += kt1 - kt0;
        return true;
    }
    __device__ int total() const {               // k-tiles of all of them
        return s.full / s.pairs * s.KT + (s.shared() ? static_cast<int>(u1 - u0) : static_cast<int>(u1) * s.KT);
    }
};

template <int BT, int BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
w8a8_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                 const __grid_constant__ CUtensorMap tmC, int c_tma, const __grid_constant__ qgi::W8A8Args a,
                 const __grid_constant__ Shares shares, float *__restrict__ P, int epi, unsigned *err,
                 uint64_t timeout_ns) {
    using G = Cfg<BT>;
    using TY = std::conditional_t<BF16 != 0, TypeBF16, TypeF16>;
    constexpr int STAGES = G::STAGES, RAWS = G::RAWS, BK = G::BK, BUFS = G::BUFS;
    constexpr uint32_t A_COLS = G::A_COLS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1024(smem_raw);
    griddep_launch_dependents();
    const uint32_t sb = smem_u32(smem);
    const uint32_t warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();      // 0 = leader
    const int pair = blockIdx.x >> 1;
    const int M = a.M, N = a.N;

    auto full_bar = [&](int s) { return sb + G::OFF_BAR + 8u * s; };
    auto empty_bar = [&](int s) { return sb + G::OFF_BAR + 8u * (STAGES + s); };
    auto raw_full = [&](int s) { return sb + G::OFF_BAR + 8u * (2 * STAGES + s); };
    auto raw_empty = [&](int s) { return sb + G::OFF_BAR + 8u * (2 * STAGES + RAWS + s); };
    auto tmem_full = [&](int b) { return sb + G::OFF_BAR + 8u * (2 * STAGES + 2 * RAWS + b); };
    auto tmem_empty = [&](int b) { return sb + G::OFF_BAR + 8u * (2 * STAGES + 2 * RAWS + BUFS + b); };
    const uint32_t drain_bar = sb + G::OFF_BAR + 8u * (2 * STAGES + 2 * RAWS + 2 * BUFS);
    volatile uint32_t *slot = reinterpret_cast<volatile uint32_t *>(smem + G::OFF_SLOT);

    // tiles: weight-row blocks of 256 (the "m" of tile_coords) x token blocks of BT
    const int tiles_w = (N + 2 * BW - 1) / (2 * BW);
    const int tiles_t = (M + BT - 1) / BT;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1 + 2 * (CONV_WARPS / G::TURNS));   // expect_tx + converters of a stage
            mbar_init(empty_bar(s), 1);                          // leader's multicast commit
        }
        for (int s = 0; s < RAWS; ++s) {
            mbar_init(raw_full(s), 1);                           // this CTA's raw weights
            mbar_init(raw_empty(s), CONV_WARPS / G::TURNS);      // its converters of a stage
        }
        for (int b = 0; b < BUFS; ++b) {
            mbar_init(tmem_full(b), 1);
            mbar_init(tmem_empty(b), 2 * EPI_WARPS);   // one lane of each epilogue warp of both CTAs
        }
        mbar_init(drain_bar, 1);
        fence_barrier_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        if (c_tma) tma_prefetch_desc(&tmC);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(const_cast<uint32_t *>(slot)), TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                   // barriers of both CTAs initialised before remote use
    tc_fence_after();
    const uint32_t tmem_base = *slot;

    if (warp == 0) {
        // ---------------------------------------------------------------- tokens' producer
        // The whole warp runs the loop and waits; one elected lane issues the copies.
        griddep_wait();                          // the tokens' halves
        uint32_t stage = 0, phase = 0;
        int issued = 0;
        bool ok = true;
        int tile, kt0, kt1, where, wb, tb;
        for (Items items(shares, pair); ok && items.next(tile, kt0, kt1, where);) {
            tile_coords(tile, tiles_w, tiles_t, wb, tb);
            const int t0 = tb * BT + static_cast<int>(rank) * (BT / 2);   // this CTA's tokens
            for (int kt = kt0; kt < kt1; ++kt) {
                // debug build: the copies' innermost coordinates are multiples of 16 bytes and begin inside K
                if (!mbar_wait_warp(empty_bar(stage), phase ^ 1, timeout_ns) ||
                    !QG_IN_BOUNDS(err, (kt * BK) % 8 == 0 && kt * BK < a.K)) {
                    ok = false;
                    break;
                }
                const uint32_t lead_full = map_to_cta(full_bar(stage), 0);
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), G::STAGE_TX);
#pragma unroll
                    for (int h = 0; h < BK / 64; ++h)   // past K's end: zeros
                        tma_load_2d_pair(sb + stage * G::X_BYTES + h * G::X_HALF, &tmX, lead_full, kt * BK + h * 64, t0);
                }
                __syncwarp();
                ++issued;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) atomicOr(err, ERR_PRODUCER);
        // no copy may land after the CTAs have left
        for (int i = max(0, issued - STAGES); rank == 0 && i < issued; ++i) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(full_bar(i % STAGES), (i / STAGES) & 1, timeout_ns))) {
                if (lane == 0) atomicOr(err, ERR_DRAIN);
                break;
            }
        }
        __syncwarp();
    } else if (warp == G::WPROD_WARP) {
        // ---------------------------------------------------------------- weights' producer
        // It need not wait for the kernel ahead, which makes the tokens' halves, touches no weights and has let this one start
        // only after all work ahead of it was done: the first weights are on their way meanwhile.
        // Weights that at most four tiles read, at nearly the same time, leave L2 first (64 x 28672 x 8192 46.9 -> 44.0 us, 64 x 16384
        // x 19456 65.9 -> 54.5, 1024 x 8192 x 28672 263 -> 252); of more, some come later (4096 x 28672 x 8192 962 -> 990).
        const uint64_t policy = tiles_t <= 4 ? l2_policy_evict_first() : l2_policy_evict_normal();
        uint32_t slot_raw = 0, phase = 0;
        int issued = 0;
        bool ok = true;
        int tile, kt0, kt1, where, wb, tb;
        for (Items items(shares, pair); ok && items.next(tile, kt0, kt1, where);) {
            tile_coords(tile, tiles_w, tiles_t, wb, tb);
            const int w0 = wb * 2 * BW + static_cast<int>(rank) * BW;     // this CTA's weights
            for (int kt = kt0; kt < kt1; ++kt) {
                if (!mbar_wait_warp(raw_empty(slot_raw), phase ^ 1, timeout_ns) ||
                    !QG_IN_BOUNDS(err, (kt * BK) % 16 == 0 && kt * BK < a.K)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    mbar_arrive_expect_tx(raw_full(slot_raw), G::RAW_BYTES);
                    tma_load_2d_hint(sb + G::OFF_RAW + slot_raw * G::RAW_BYTES, &tmW, raw_full(slot_raw), kt * BK, w0, policy);
                }
                __syncwarp();
                ++issued;
                if (++slot_raw == RAWS) {
                    slot_raw = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok && lane == 0) atomicOr(err, ERR_PRODUCER);
        for (int i = max(0, issued - RAWS); i < issued; ++i) {
            if (!mbar_wait_warp(raw_full(i % RAWS), (i / RAWS) & 1, timeout_ns)) {
                if (lane == 0) atomicOr(err, ERR_DRAIN);
                break;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // --------------------------------------------------------- MMA issuer
            const uint64_t bdesc0 = smem_desc(sb, 16, 1024, SWZ_128B);
            uint32_t buf = 0, acc_phase = 0, stage = 0, phase = 0;
            bool ok = true;
            int tile, kt0, kt1, where;
            for (Items items(shares, pair); ok && items.next(tile, kt0, kt1, where);) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(tmem_empty(buf), acc_phase ^ 1, timeout_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int kt = kt0; kt < kt1; ++kt) {
                    if (!mbar_wait_warp(full_bar(stage), phase, timeout_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_col = tmem_base + G::A_COL0 + stage * A_COLS;
                    const uint64_t bdesc = bdesc0 + stage * (G::X_BYTES >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t j = 0; j < BK / 16; ++j)
                            mma_f16_pair_ta(tmem_base + buf * BT, a_col + 8 * j, bdesc + (j / 4) * (G::X_HALF >> 4) + 2 * (j % 4),
                                            G::IDESC, kt > kt0 || j > 0 ? 1u : 0u);
                        tc_commit_pair(empty_bar(stage), 3);
                    }
                    __syncwarp();
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair(tmem_full(buf), 3);
                __syncwarp();
                if (++buf == BUFS) {
                    buf = 0;
                    acc_phase ^= 1;
                }
            }
            if (elect_one()) {
                if (!ok) atomicOr(err, ERR_MMA);
                tc_commit_pair(drain_bar, 3);
            }
        }
        __syncwarp();
        // both CTAs: every pair MMA writing this CTA's TMEM has completed before it is freed
        if (!mbar_wait(drain_bar, 0, timeout_ns) && lane == 0) atomicOr(err, ERR_DRAIN);
    } else if (warp >= CONV_WARP0) {
        // ----------------------------------------------------------------- converters
        // Lane i of a warp of lane quarter q converts weight row 32 q + i of this CTA's 128, 64 k at a time.
        const uint32_t q = warp & 3;
        const int which = static_cast<int>(warp - CONV_WARP0) >> 2;      // of the quarter's two warps
        const int first = G::TURNS == 2 ? which : 0;
        const uint32_t h = G::TURNS == 2 ? 0 : which;
        const uint32_t lead_full = map_to_cta(full_bar(0), 0);
        const uint32_t r = q * 32 + lane;
        const int total = Items(shares, pair).total();
        uint32_t stage = static_cast<uint32_t>(first), phase = 0, slot_raw = stage, phase_raw = 0;
        const uint8_t *row = smem + G::OFF_RAW + r * BK;
        // TMA's swizzle: chunk c of row r lies at c ^ (r % 8) of 128 bytes, or c ^ (r / 2 % 4) of 64
        const uint32_t swz = BK == 128 ? r & 7 : (r >> 1) & 3;
        // A wait that gave up leaves the others no time: the lanes stay together (a vote after each wait costs 64 and 128 tokens 10
        // to 20 %), and the warp goes through its k-tiles at once, whatever they hold.
        uint64_t limit = timeout_ns;
        for (int i = first; i < total; i += G::TURNS) {
            if (!mbar_wait(raw_full(slot_raw), phase_raw, limit)) limit = 0;
            const uint8_t *raw = row + slot_raw * G::RAW_BYTES;
            uint32_t out[32];
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) {
                const uint4 d = *reinterpret_cast<const uint4 *>(raw + (((4 * h + c) ^ swz) << 4));
                i8x4_to_f16(d.x, out[8 * c], out[8 * c + 1]);
                i8x4_to_f16(d.y, out[8 * c + 2], out[8 * c + 3]);
                i8x4_to_f16(d.z, out[8 * c + 4], out[8 * c + 5]);
                i8x4_to_f16(d.w, out[8 * c + 6], out[8 * c + 7]);
            }
            // read through the generic proxy, written next by TMA through the async proxy
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(raw_empty(slot_raw));
            // the MMAs that last read this TMEM slot have completed
            if (!mbar_wait(empty_bar(stage), phase ^ 1, limit)) limit = 0;
            tc_fence_after();
            tmem_st_32x32b_x32(tmem_base + ((q * 32) << 16) + G::A_COL0 + stage * A_COLS + 32 * h, out);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed_cluster(lead_full + 8u * stage);
            if ((stage += G::TURNS) >= STAGES) {
                stage -= STAGES;
                phase ^= 1;
            }
            if ((slot_raw += G::TURNS) >= RAWS) {
                slot_raw -= RAWS;
                phase_raw ^= 1;
            }
        }
        if (__any_sync(0xFFFFFFFFu, limit == 0) && lane == 0) atomicOr(err, ERR_PRODUCER);
    } else {
        // ---------------------------------------------------------------- epilogue
        // Lane i of a warp of lane quarter q holds output column n = weight row 32 q + i; the warp covers
        // BT / 2 of the tile's tokens, 32 per TMEM read.
        const uint32_t q = warp & 3;
        const uint32_t half = (warp - 2) >> 2;
        const uint32_t lead_empty = map_to_cta(tmem_empty(0), 0);
        const uint32_t stg = sb + G::OFF_EPI + (warp - 2) * G::EPI_BYTES;
        float *sa_room = reinterpret_cast<float *>(smem + G::OFF_SA) + (warp - 2) * (BT / 2);
        uint32_t buf = 0, acc_phase = 0;
        griddep_wait();
        int tile, kt0, kt1, where, wb, tb;
        for (Items items(shares, pair); items.next(tile, kt0, kt1, where);) {
            tile_coords(tile, tiles_w, tiles_t, wb, tb);
            const int n0 = wb * 2 * BW + static_cast<int>(rank) * BW + static_cast<int>(q * 32);
            const int n = n0 + static_cast<int>(lane);
            const int m0 = tb * BT + static_cast<int>(half) * (BT / 2);
            float sw = 0.0f, bias = 0.0f;        // while the tile's MMAs run
            if (n < N) {
                sw = __ldg(a.sw + n);
                if (a.bias) bias = load_16(a.bias, n, BF16);
            }
            __syncwarp();
            for (int c = static_cast<int>(lane); c < BT / 2; c += 32) sa_room[c] = m0 + c < M ? __ldg(a.sa + m0 + c) : 0.0f;
            __syncwarp();
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_sleep(tmem_full(buf), acc_phase, timeout_ns, 128))) {
                if (lane == 0) atomicOr(err, ERR_EPILOGUE);
                break;
            }
            tc_fence_after();
            if (c_tma) {                         // the previous tile's stores have finished reading the staging
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
            }
            const uint32_t d_col = tmem_base + ((q * 32) << 16) + buf * BT + half * (BT / 2), release = lead_empty + 8 * buf;
            if (++buf == BUFS) {
                buf = 0;
                acc_phase ^= 1;
            }
#pragma unroll 1
            for (int ch = 0; ch < G::CHUNKS; ++ch) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(d_col + ch * 32, v);
                tmem_wait_ld();
                if (ch == G::CHUNKS - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_relaxed_cluster(release);
                }
                const int mc = m0 + ch * 32;
                if (where >= 0) {
                    if (!QG_IN_BOUNDS(err, where < 2 * shares.sharers && shares.shared() && half * (BT / 2) + ch * 32 + 32 <= BT)) continue;
                    // this range's sums, [token of the tile][weight row of the tile]: a store writes 32 consecutive floats
                    float *pl = P + (int64_t(where) * BT + half * (BT / 2) + ch * 32) * (2 * BW) + rank * BW + q * 32 + lane;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (mc + c < M) pl[c * (2 * BW)] = __uint_as_float(v[c]);
                } else if (c_tma) {
                    // row c of the chunk: token mc + c, columns n0 .. n0 + 31
                    const uint32_t to = stg + ch * 2048 + lane * 2;
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 sa = *reinterpret_cast<const float4 *>(sa_room + ch * 32 + c);
                        float x[4];
                        scaled2(x[0], x[1], __uint_as_float(v[c]), __uint_as_float(v[c + 1]), sa.x, sa.y, sw, bias);
                        scaled2(x[2], x[3], __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]), sa.z, sa.w, sw, bias);
                        if (epi & qgi::EPI_RELU) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[j] = fmaxf(x[j], 0.0f);
                        }
                        const uint32_t lo = TY::pack(x[0], x[1]), hi = TY::pack(x[2], x[3]);
                        st_shared_u16(to + c * 64, static_cast<uint16_t>(lo));
                        st_shared_u16(to + (c + 1) * 64, static_cast<uint16_t>(lo >> 16));
                        st_shared_u16(to + (c + 2) * 64, static_cast<uint16_t>(hi));
                        st_shared_u16(to + (c + 3) * 64, static_cast<uint16_t>(hi >> 16));
                    }
                } else if (n < N) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if (mc + c >= M || !QG_IN_BOUNDS(err, mc + c >= 0 && n >= 0)) continue;
                        uint16_t *dst = static_cast<uint16_t *>(a.C) + (mc + c) * a.ldc + n;
                        const float old = epi & qgi::EPI_ACCUMULATE ? load_16(dst, 0, BF16) : 0.0f;
                        *dst = round_16(finish(__uint_as_float(v[c]), sa_room[ch * 32 + c], sw, bias, old, epi), BF16);
                    }
                }
            }
            if (c_tma && where < 0) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int ch = 0; ch < G::CHUNKS; ++ch)   // blocks wholly past M or N are not stored
                        if (n0 < N && m0 + ch * 32 < M && QG_IN_BOUNDS(err, n0 >= 0 && n0 % 8 == 0 && m0 >= 0)) tma_store_2d(&tmC, stg + ch * 2048, n0, m0 + ch * 32);
                    bulk_commit();
                }
            }
        }
        if (c_tma && lane == 0) bulk_wait_all();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();                   // no remote arrival or multicast targets an exited CTA
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// The tokens' codes as halves, rows of `ldh` (K rounded up to 16, at least): 16 codes a thread.
__global__ void __launch_bounds__(256) codes_to_f16_kernel(const int8_t *__restrict__ A, int64_t lda, int M, int K,
                                                           uint16_t *__restrict__ H, int64_t ldh, unsigned *err) {
    griddep_wait();
    griddep_launch_dependents();                                   // after the wait: see the pair kernel's early copies
    const int per_row = (K + 15) / 16;
    const int64_t total = static_cast<int64_t>(M) * per_row;
    for (int64_t i = blockIdx.x * int64_t(256) + threadIdx.x; i < total; i += gridDim.x * int64_t(256)) {
        const int64_t m = i / per_row;
        const int k = static_cast<int>(i - m * per_row) * 16;
        const int8_t *src = A + m * lda + k;
        uint4 d;
        if (k + 16 <= K) {
            d = __ldg(reinterpret_cast<const uint4 *>(src));
        } else {                                                   // a row's end: only its own bytes
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (k + j < K) w[j / 4] |= uint32_t(uint8_t(__ldg(src + j))) << (8 * (j & 3));
            d = make_uint4(w[0], w[1], w[2], w[3]);
        }
        uint32_t o[8];
        i8x4_to_f16(d.x, o[0], o[1]);
        i8x4_to_f16(d.y, o[2], o[3]);
        i8x4_to_f16(d.z, o[4], o[5]);
        i8x4_to_f16(d.w, o[6], o[7]);
        uint4 *dst = reinterpret_cast<uint4 *>(H + m * ldh + k);
        if (!QG_IN_BOUNDS(err, m < M && k < K && k + 16 <= ldh)) continue;
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// The tiles that several pairs shared, from their partial sums in the order of K: `parts` blocks a tile, four columns a
// thread, four tokens' rows of 256 columns at a time.  What goes by tile or column is found once a block.
template <int BT>
__global__ void __launch_bounds__(256) w8a8_reduce_kernel(const float *__restrict__ P, const __grid_constant__ Shares shares,
                                                          const __grid_constant__ qgi::W8A8Args a, int parts, int vec, int epi, unsigned *err) {
    griddep_launch_dependents();
    constexpr int64_t SLOT = int64_t(BT) * (2 * BW);
    const int t = blockIdx.x / parts, part = blockIdx.x - t * parts;
    const int p0 = shares.owner(t * shares.KT), p1 = shares.owner((t + 1) * shares.KT - 1);
    int wb, tb;
    tile_coords(shares.full + t, (a.N + 2 * BW - 1) / (2 * BW), (a.M + BT - 1) / BT, wb, tb);
    const int col = 4 * static_cast<int>(threadIdx.x & 63), n = wb * 2 * BW + col;
    // piece p of the tile is the first of its pair's range where that begins inside the tile or at its start: all but p0's may
    const float *first = P + (2 * p0 + (shares.begin(p0) >= uint32_t(t) * shares.KT ? 0 : 1)) * SLOT + col, *others = P + col;
    if (p0 == p1 || n >= a.N) return;            // a whole tile, written by its pair
    if (!QG_IN_BOUNDS(err, t < shares.rest && p0 >= 0 && p0 < p1 && p1 < shares.sharers)) return;
    griddep_wait();
    float sw[4], bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        sw[j] = n + j < a.N ? __ldg(a.sw + n + j) : 0.0f;
        bias[j] = a.bias && n + j < a.N ? load_16(a.bias, n + j, a.bf16) : 0.0f;
    }
    const bool whole = vec && n + 4 <= a.N;
    for (int token = 4 * part + static_cast<int>(threadIdx.x >> 6); token < BT; token += 4 * parts) {
        const int64_t m = int64_t(tb) * BT + token;
        if (m >= a.M || !QG_IN_BOUNDS(err, m >= 0 && token < BT && n >= 0)) break;
        const int row = token * (2 * BW);
        float4 sum = __ldcg(reinterpret_cast<const float4 *>(first + row));
        for (int p = p0 + 1; p <= p1; p += 8) {  // eight pieces' loads at once, whatever is left of them
            float4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = p + j <= p1 ? __ldcg(reinterpret_cast<const float4 *>(others + 2 * (p + j) * SLOT + row))
                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum.x += v[j].x, sum.y += v[j].y, sum.z += v[j].z, sum.w += v[j].w;
        }
        const float sa = __ldg(a.sa + m), sums[4] = {sum.x, sum.y, sum.z, sum.w};
        uint16_t *dst = static_cast<uint16_t *>(a.C) + m * a.ldc + n;
        uint16_t out[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n + j >= a.N) break;
            const float old = epi & qgi::EPI_ACCUMULATE ? load_16(dst, j, a.bf16) : 0.0f;
            out[j] = round_16(finish(sums[j], sa, sw[j], bias[j], old, epi), a.bf16);
            if (!whole) dst[j] = out[j];
        }
        if (whole) *reinterpret_cast<uint2 *>(dst) = make_uint2(out[0] | uint32_t(out[1]) << 16, out[2] | uint32_t(out[3]) << 16);
    }
}

// How the tiles left after whole waves are cut: not at all; each into the same number of pieces; or all together into equal
// ranges, which keeps every pair busy but leaves pieces of two tiles to most, and so more partial sums.
enum Cut { NONE, EVEN, EQUAL };

struct Plan {
    int bt;
    Cut cut;
    Shares shares;
};

int k_of(int bt) { return bt == 256 ? Cfg<256>::BK : Cfg<64>::BK; }

// Work of M tokens in tiles of bt.
Shares share(int bt, Cut cut, int M, int N, int K, int num_sms) {
    Shares s;
    const int bk = k_of(bt);
    s.KT = (K + bk - 1) / bk;
    const int most = std::max(1, num_sms / 2);
    const int64_t tiles = int64_t((N + 2 * BW - 1) / (2 * BW)) * ((M + bt - 1) / bt);
    s.pairs = most;
    s.full = static_cast<int>(tiles / most * most);
    s.rest = static_cast<int>(tiles - s.full);
    s.sharers = s.rest;
    if (cut != NONE && s.rest > 0) {
        // ranges of at least 256 of K, about 8 a tile at most (more cost the reduction a second round of loads)
        int64_t most_shares = std::min<int64_t>({most, int64_t(s.rest) * s.KT * bk / 256, int64_t(s.rest) * 8});
        if (cut == EVEN) most_shares -= most_shares % s.rest;
        if (most_shares > s.rest && int64_t(s.rest) * s.KT * most_shares < (int64_t(1) << 31)) s.sharers = static_cast<int>(most_shares);
    }
    if (s.full == 0) s.pairs = s.sharers;
    return s;
}

// Estimated us of a plan: the waves' walks over K, what stays open at a tile's end, the reduction's launch and traffic.
// Measured: a k-tile takes a pair 0.29, 0.34 and 0.30 us (64, 128 and 128 k for 256, 128 and 64 tokens; matrices that stay in L2);
// a wave of 256-token tiles, with one accumulator, ends 2.8 us after its walk, of smaller ones 0.2 (1.5 the last); all pairs together
// get 6.3 TB/s of weights from memory, which each weight leaves once however many token tiles meet it; partial sums are written and
// read at 5 TB/s.
double cost(int bt, const Shares &s, int M, int K) {
    const double per_kt = bt == 256 ? 0.29 : bt == 128 ? 0.34 : 0.30, ends = bt == 256 ? 2.8 : 0.2;
    const double tile_us = double(2 * BW) * K / ((M + bt - 1) / bt) / 6.3e6;           // a tile's weights from memory
    const int waves = s.pairs ? s.full / s.pairs : 0;
    double us = waves * (std::max(s.KT * per_kt, s.pairs * tile_us) + ends);
    if (s.rest) us += std::max(double(s.rest) * s.KT / s.sharers * per_kt, s.rest * tile_us) + ends;
    if (bt < 256) us += 1.3;
    if (s.shared()) us += 2.0 + 2.0 * (s.sharers + (s.sharers % s.rest ? s.rest : 0)) * bt * (2 * BW) * 4 / 5e6;
    return us;
}

Plan choose(int M, int N, int K, int num_sms) {
    Plan best{};
    double least = 1e300;
    for (int bt : {256, 128, 64})
        for (Cut cut : {NONE, EVEN, EQUAL}) {
            const Shares s = share(bt, cut, M, N, K, num_sms);
            const double us = cost(bt, s, M, K);
            if (us < least) {
                least = us;
                best = {bt, cut, s};
            }
        }
    return best;
}

template <int BT>
cudaError_t launch_bt(const qgi::W8A8Args &a, const CUtensorMap &tmX, const CUtensorMap &tmW, const CUtensorMap &tmC,
                      int c_tma, const Shares &shares, float *P, const qgi::LaunchCtx &ctx) {
    auto kern = a.bf16 ? w8a8_pair_kernel<BT, 1> : w8a8_pair_kernel<BT, 0>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BT>::SMEM);
    if (e == cudaSuccess)
        e = launch_dependent(kern, dim3(2 * shares.pairs), THREADS, Cfg<BT>::SMEM, ctx.stream, tmX, tmW, tmC, c_tma, a, shares, P,
                             ctx.epi, ctx.err, ctx.timeout_ns);
    if (e == cudaSuccess && shares.shared()) {
        const int vec = reinterpret_cast<uintptr_t>(a.C) % 8 == 0 && a.ldc % 4 == 0;
        const int parts = std::max(1, std::min(BT / 4, (4 * ctx.num_sms + shares.rest - 1) / shares.rest));
        e = launch_dependent(w8a8_reduce_kernel<BT>, dim3(shares.rest * parts), 256, 0, ctx.stream, P, shares, a, parts, vec, ctx.epi, ctx.err);
    }
    return e;
}

unsigned grid_for(int64_t threads, const qgi::LaunchCtx &ctx) {
    return static_cast<unsigned>(std::min<int64_t>((threads + 255) / 256, 8 * ctx.num_sms));
}

}  // namespace

namespace qgi {

// A product of many tokens is taken in slices of rows, so that the tokens' halves never hold more scratch than this.
constexpr int64_t SLICE_BYTES = int64_t(1) << 29;

static cudaError_t launch_slice(const W8A8Args &a, uint16_t *H, int64_t ldh, float *P, int bt, const Shares &shares,
                                const CUtensorMap &tmW, const LaunchCtx &ctx, bool *encode_ok) {
    // Output through TMA stores where C allows a tensor map.  They write whole 16-byte units, past a row's end too
    // where N is no multiple of 8 (measured); accumulating reads the old C: direct stores in both cases.
    const int c_tma = reinterpret_cast<uintptr_t>(a.C) % 16 == 0 && a.ldc % 8 == 0 && a.N % 8 == 0 &&
                      a.ldc < (int64_t(1) << 39) && !(ctx.epi & EPI_ACCUMULATE);
    CUtensorMap tmX, tmC;
    *encode_ok = encode_tma_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, H, a.K, a.M, ldh * 2, 64, bt / 2,
                               CU_TENSOR_MAP_SWIZZLE_128B);
    if (*encode_ok && c_tma)
        *encode_ok = encode_tma_2d(&tmC, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.C, a.N, a.M, a.ldc * 2, 32, 32,
                                   CU_TENSOR_MAP_SWIZZLE_NONE);
    else
        tmC = tmX;   // unused
    if (!*encode_ok) return cudaErrorInvalidValue;
    cudaError_t e = launch_dependent(codes_to_f16_kernel, dim3(grid_for(a.M * int64_t((a.K + 15) / 16), ctx)), 256, 0,
                                     ctx.stream, a.A, a.lda, a.M, a.K, H, ldh, ctx.err);
    if (e == cudaSuccess)
        e = bt == 64    ? launch_bt<64>(a, tmX, tmW, tmC, c_tma, shares, P, ctx)
            : bt == 128 ? launch_bt<128>(a, tmX, tmW, tmC, c_tma, shares, P, ctx)
                        : launch_bt<256>(a, tmX, tmW, tmC, c_tma, shares, P, ctx);
    return e;
}

cudaError_t launch_w8a8_pair(const W8A8Args &a, const LaunchCtx &ctx, bool *encode_ok) {
    const int64_t ldh = (a.K + 63) / 64 * int64_t(64);
    const int slice = static_cast<int>(std::min<int64_t>(a.M, std::max<int64_t>(SLICE_BYTES / (2 * ldh) / 256 * 256, 256)));
    const Plan plan = choose(slice, a.N, a.K, ctx.num_sms);
    const int bt = plan.bt, bk = k_of(bt);
    const Shares &shares = plan.shares;
    const Shares last = a.M % slice ? share(bt, plan.cut, a.M % slice, a.N, a.K, ctx.num_sms) : shares;
    const size_t x_bytes = (static_cast<size_t>(slice) * ldh * 2 + 255) / 256 * 256;
    const bool shared = shares.shared() || last.shared();
    const size_t p_bytes = shared ? static_cast<size_t>(std::max(shares.sharers, last.sharers)) * 2 * bt * (2 * BW) * 4 : 0;
    CUtensorMap tmW;
    *encode_ok = encode_tma_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.W, a.K, a.N, a.ldw, bk, BW,
                               bk == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
    if (!*encode_ok) return cudaErrorInvalidValue;
    void *ws = nullptr;
    cudaError_t e = scratch_alloc(x_bytes + p_bytes, ctx, &ws);
    if (e != cudaSuccess) return e;
    uint8_t *base = static_cast<uint8_t *>(ws);
    for (int64_t m0 = 0; m0 < a.M && e == cudaSuccess; m0 += slice) {
        W8A8Args part = a;
        part.A += m0 * a.lda;
        part.sa += m0;
        part.C = static_cast<uint16_t *>(a.C) + m0 * a.ldc;
        part.M = static_cast<int>(std::min<int64_t>(slice, a.M - m0));
        e = launch_slice(part, reinterpret_cast<uint16_t *>(base), ldh, reinterpret_cast<float *>(base + x_bytes), bt,
                         part.M == slice ? shares : last, tmW, ctx, encode_ok);
    }
    const cudaError_t f = scratch_free(ws, ctx);
    return e != cudaSuccess ? e : f;
}

}  // namespace qgi

// w8a8_decode.cu -- product of 8-bit integers for a few tokens, bound by the weights' bytes.
//
// A weight stream: a producer warp keeps STAGES boxes of 16 NF weight rows x 128 bytes of K in flight by TMA, with the
// same 128 bytes of the tokens' rows beside each.  Four consumer warps take 32 k of a stage each, for all its rows:
// per 16-row fragment a lane quad turns 8 consecutive int8 of rows g and g + 8 into halves (exact) and feeds two
// mma.sync m16n8k16, weights as the 16-row operand and tokens as the 8-column operand; the 32 k are permuted alike for both, so the sums
// are unchanged.  Sums are fp32 over the whole of K, scaled once at the end.
//
// A block of rows is a cluster's: where there are few blocks of rows, its K is cut over the cluster's CTAs, whose
// sums meet through distributed shared memory (no scratch, no second launch).  Partial sums are added in the order of
// ranks and warps, so results repeat bit for bit.
//
// Bound by the weights' bytes: 1 x 28672 x 8192 36 us (6.5 TB/s), 1 x 8192 x 28672 37.9, 8 x 16384 x 19456 50.8 (6.3 TB/s); at 16 tokens
// the tokens' rows, read again for every block of rows, add 5 to 12 % (39 and 42.6 us); small matrices by start and end: 4096 x
// 4096 6.6 us for 1 token, 7.1 for 8, where the bytes take 2.5 (a cluster's start and its two meetings, the first copies' latency).
// mma.sync is 17 % busy at 8 tokens.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "qgemm_common.cuh"
#include "w8a8_common.cuh"

namespace {

using namespace qg;

constexpr int CONSUMERS = 4;
constexpr int THREADS = (CONSUMERS + 1) * 32;
constexpr int KC = 128;                     // bytes of K per stage

// NH: 8-token columns (M <= 8 NH); NF: 16-row weight fragments of a block of rows.
template <int NH, int NF, int STAGES_>
struct Cfg {
    static constexpr int STAGES = STAGES_;
    static constexpr int ROWS = 16 * NF;
    static constexpr uint32_t W_BYTES = ROWS * KC;
    static constexpr uint32_t X_BYTES = 8 * NH * KC;
    static constexpr uint32_t STAGE = W_BYTES + X_BYTES;
    static constexpr uint32_t RED = CONSUMERS * NF * NH * 4 * 32 * 4;   // sums of the warps: [warp][NF][NH][4][lane]
    static constexpr uint32_t OFF_BAR = STAGES * STAGE;
    static constexpr uint32_t OFF_RED = OFF_BAR + 2 * STAGES * 8;
    // Where K is cut a CTA has one block of rows, and its sums take the stages' place: a fourth CTA an SM at 16 tokens (8192 x
    // 28672 45.6 -> 42.5 us).
    static constexpr uint32_t smem(int splits) { return 1024 + (splits > 1 ? OFF_RED : OFF_RED + RED); }
    static_assert(RED <= OFF_BAR, "sums in the stages' place");
    static_assert(STAGE % 1024 == 0, "stages stay 1 KB aligned for the 128-byte swizzle");
};

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

// One stage's products: this warp's 32 k of every row.
template <int NH, int NF>
__device__ __forceinline__ void stage_math(float (&acc)[NF][NH][4], const uint8_t *st, uint32_t off) {
    uint32_t x[NH][4];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        const uint2 v = *reinterpret_cast<const uint2 *>(st + 16 * NF * KC + h * 1024 + off);
        i8x4_to_f16(v.x, x[h][0], x[h][1]);
        i8x4_to_f16(v.y, x[h][2], x[h][3]);
    }
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const uint2 wa = *reinterpret_cast<const uint2 *>(st + off + f * 2048);
        const uint2 wb = *reinterpret_cast<const uint2 *>(st + off + f * 2048 + 1024);
        uint32_t a0[4], a1[4];
        i8x4_to_f16(wa.x, a0[0], a0[2]);
        i8x4_to_f16(wb.x, a0[1], a0[3]);
        i8x4_to_f16(wa.y, a1[0], a1[2]);
        i8x4_to_f16(wb.y, a1[1], a1[3]);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            mma_16816(acc[f][h], a0, x[h][0], x[h][1], acc[f][h]);
            mma_16816(acc[f][h], a1, x[h][2], x[h][3], acc[f][h]);
        }
    }
}

template <int NH, int NF, int STAGES_>
__global__ void __launch_bounds__(THREADS)
w8a8_decode_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ qgi::W8A8Args a, int splits, int epi, unsigned *err, uint64_t timeout_ns) {
    using G = Cfg<NH, NF, STAGES_>;
    constexpr int STAGES = G::STAGES, ROWS = G::ROWS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_1024(smem_raw);
    griddep_launch_dependents();
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto full_bar = [&](int s) { return sb + G::OFF_BAR + 8u * s; };
    auto empty_bar = [&](int s) { return sb + G::OFF_BAR + 8u * (STAGES + s); };
    const uint32_t off_red = splits > 1 ? 0 : G::OFF_RED;
    float *red = reinterpret_cast<float *>(smem + off_red);

    const int nrb = (a.N + ROWS - 1) / ROWS;     // blocks of rows
    const int nkc = (a.K + KC - 1) / KC;         // stages of all of K
    const int rank = splits > 1 ? static_cast<int>(blockIdx.x) % splits : 0;
    const int kc0 = static_cast<int>(int64_t(nkc) * rank / splits), kc1 = static_cast<int>(int64_t(nkc) * (rank + 1) / splits);
    const int first = static_cast<int>(blockIdx.x) / splits, step = static_cast<int>(gridDim.x) / splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), CONSUMERS);
        }
        fence_barrier_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    __syncthreads();
    griddep_wait();

    if (warp == CONSUMERS) {
        // ------------------------------------------------------------------- producer
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            int issued = 0;
            bool ok = true;
            const uint64_t stream_once = l2_policy_evict_first();   // the weights are read once
            for (int rb = first; rb < nrb && ok; rb += step) {
                for (int kc = kc0; kc < kc1; ++kc) {
                    // debug build: innermost coordinates multiples of 16 bytes, the box begins inside the planes
                    if (!mbar_wait(empty_bar(stage), phase ^ 1, timeout_ns) ||
                        !QG_IN_BOUNDS(err, (kc * KC) % 16 == 0 && kc * KC < a.K && rb * ROWS < a.N)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = sb + stage * G::STAGE;
                    mbar_arrive_expect_tx(full_bar(stage), G::STAGE);
                    tma_load_2d_hint(st, &tmW, full_bar(stage), kc * KC, rb * ROWS, stream_once);
                    tma_load_2d(st + G::W_BYTES, &tmX, full_bar(stage), kc * KC, 0);
                    ++issued;
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) atomicOr(err, ERR_PRODUCER);
            for (int i = max(0, issued - STAGES); i < issued; ++i)
                if (!mbar_wait(full_bar(i % STAGES), (i / STAGES) & 1, timeout_ns)) {
                    atomicOr(err, ERR_DRAIN);
                    break;
                }
        }
        __syncwarp();
        if (splits > 1) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    // ---------------------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    // bytes 32 w + 8 t .. + 8 of row g (the 128-byte swizzle: chunk c of row r at c ^ (r % 8)); row g + 8 is 1 KB on
    const uint32_t off = static_cast<uint32_t>(g) * 128 +
                         ((static_cast<uint32_t>(2 * warp + (t >> 1)) ^ static_cast<uint32_t>(g)) << 4) +
                         static_cast<uint32_t>((t & 1) * 8);
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int rb = first; rb < nrb; rb += step) {
        float acc[NF][NH][4];
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[f][h][i] = 0.0f;
        for (int kc = kc0; kc < kc1 && ok; kc += 2) {
            // two stages at a time: twice the independent work between waits
            const bool two = kc + 1 < kc1;
            uint32_t stage2 = stage + 1, phase2 = phase;
            if (stage2 == STAGES) {
                stage2 = 0;
                phase2 ^= 1;
            }
            if (!mbar_wait_warp(full_bar(stage), phase, timeout_ns) ||
                (two && !mbar_wait_warp(full_bar(stage2), phase2, timeout_ns))) {
                if (lane == 0) atomicOr(err, ERR_EPILOGUE);
                ok = false;
                break;
            }
            stage_math<NH, NF>(acc, smem + stage * G::STAGE, off);
            if (two) stage_math<NH, NF>(acc, smem + stage2 * G::STAGE, off);
            // read through the generic proxy, written next by TMA through the async proxy
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(empty_bar(stage));
                if (two) mbar_arrive(empty_bar(stage2));
            }
            stage = two ? (stage2 + 1 == STAGES ? 0 : stage2 + 1) : stage2;
            phase = two ? (stage2 + 1 == STAGES ? phase2 ^ 1 : phase2) : phase2;
        }
        if (splits > 1) asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory");   // every warp has read its stages
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) red[(((warp * NF + f) * NH + h) * 4 + i) * 32 + lane] = acc[f][h][i];
        asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory");
        // the four warps' sums, an output a thread: column r of the block of token m
        auto place = [&](int m, int r) {
            return (((r >> 4) * NH + (m >> 3)) * 4 + ((r >> 3) & 1) * 2 + (m & 1)) * 32 + (r & 7) * 4 + ((m & 7) >> 1);
        };
        auto store = [&](int m, int n, float sum) {
            if (!QG_IN_BOUNDS(err, m >= 0 && m < a.M && n >= 0 && n < a.N)) return;
            uint16_t *dst = static_cast<uint16_t *>(a.C) + m * a.ldc + n;
            const float bias = a.bias ? load_16(a.bias, n, a.bf16) : 0.0f;
            const float old = epi & qgi::EPI_ACCUMULATE ? load_16(dst, 0, a.bf16) : 0.0f;
            *dst = round_16(finish(sum, __ldg(a.sa + m), __ldg(a.sw + n), bias, old, epi), a.bf16);
        };
        constexpr int WARP_SUMS = NF * NH * 4 * 32;
        for (int i = static_cast<int>(threadIdx.x); i < ROWS * a.M; i += CONSUMERS * 32) {
            const int m = i / ROWS, r = i - m * ROWS, at = place(m, r);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < CONSUMERS; ++w) sum += red[w * WARP_SUMS + at];
            if (splits > 1) red[at] = sum;       // its own place: no other output reads it
            else if (rb * ROWS + r < a.N) store(m, rb * ROWS + r, sum);
        }
        if (splits > 1) {                        // one block of rows a cluster: its CTAs' sums, an output a thread of the cluster
            cluster_sync();
            for (int i = rank * CONSUMERS * 32 + static_cast<int>(threadIdx.x); i < ROWS * a.M; i += splits * CONSUMERS * 32) {
                const int m = i / ROWS, r = i - m * ROWS, n = rb * ROWS + r;
                const uint32_t addr = sb + off_red + 4u * place(m, r);
                float part[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) part[c] = c < splits ? ld_cluster(map_to_cta(addr, c)) : 0.0f;
                float sum = 0.0f;
#pragma unroll
                for (int c = 0; c < 8; ++c) sum += part[c];
                if (n < a.N) store(m, n, sum);
            }
            cluster_sync();                      // no CTA leaves while another reads its sums
            return;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS * 32) : "memory");
    }
}

constexpr uint32_t SM_SMEM = 233472;            // shared memory of an SM, 1 KB of it each CTA's own

// How the work is laid out: NF fragments of 16 rows a block, K over `splits` CTAs, and its estimated us.
struct Layout {
    int splits;
    int64_t grid;
    double us;
};

// The best split for one block height.  Measured on 27 products (1, 8 and 16 tokens, nine matrices from 2048 x 8192 to 16384 x 19456, every
// height and split; the rule's choice is 0.2 % behind the fastest on average, 2.2 % at most): an SM takes 5 + 0.63 KB^-1 x (its KB
// of weights on their way) bytes a ns of its own share, tokens' rows count 1.3 times; all together at most 6.5 TB/s; both bound at once
// cost more than either (a fourth-power mean); a cluster costs its start and meetings.  One block of rows a cluster, all of
// them at once (clusters of other than 2, 4 or 8 leave room unused: 602 CTAs in clusters of 7 ran in two rounds where 608
// fit), or with K whole as many as there are.  Lower blocks count 1.2 % for each fragment less: their clusters find places less evenly.
template <class G>
Layout layout(const qgi::W8A8Args &a, int num_sms) {
    const int64_t nrb = (int64_t(a.N) + G::ROWS - 1) / G::ROWS;
    const int nkc = (a.K + KC - 1) / KC;
    Layout best{1, 1, 1e300};
    for (int s = 1; s <= 8; ++s) {
        if (nkc < 2 * s && s > 1) break;
        const int per_sm = std::max(1, int(SM_SMEM / (G::smem(s) + 1024)));
        const int64_t room = int64_t(num_sms) * per_sm;
        if (s > 1 && nrb * s > (s & (s - 1) ? room * 17 / 20 : room)) continue;
        const int64_t ctas = std::min(nrb * s, room), rounds = (nrb * s + ctas - 1) / ctas;
        const int64_t each = (ctas + num_sms - 1) / num_sms * rounds;                  // on the fullest SM
        const double rate = 5.0 + 0.63 * double(std::min<int64_t>(each, per_sm) * G::STAGES * G::W_BYTES) / 1024;
        const double own = double(each) * (G::W_BYTES + 1.3 * G::X_BYTES) * ((nkc + s - 1) / s) / 1e3 / rate;
        const double all = double(a.N) * a.K / 6.5e6, own2 = own * own, all2 = all * all;
        const double us = (std::sqrt(std::sqrt(own2 * own2 + all2 * all2)) + (s > 1 ? 0.9 + 0.15 * s * (1.0 + a.M / 8.0) : 0.0)) *
                          (1.0 + 0.012 * (4 - G::ROWS / 16));
        if (us < best.us) best = {s, ctas, us};
    }
    return best;
}

template <int NH, int NF, int STAGES>
cudaError_t launch_nh(const qgi::W8A8Args &a, const Layout &l, const qgi::LaunchCtx &ctx, bool *encode_ok) {
    using G = Cfg<NH, NF, STAGES>;
    CUtensorMap tmW, tmX;
    *encode_ok =
        qgi::encode_tma_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.W, a.K, a.N, a.ldw, KC, G::ROWS, CU_TENSOR_MAP_SWIZZLE_128B) &&
        qgi::encode_tma_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.A, a.K, a.M, a.lda, KC, 8 * NH, CU_TENSOR_MAP_SWIZZLE_128B);
    if (!*encode_ok) return cudaErrorInvalidValue;
    auto kern = w8a8_decode_kernel<NH, NF, STAGES>;
    constexpr uint32_t MOST = 232448;            // of a CTA
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(l.grid));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = ctx.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(l.splits);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // CTAs spread evenly: each takes the shared memory that leaves no room for more on its SM than there are on the fullest (8 x
    // 4096 x 4096, 512 CTAs: 7.1 us against 7.7 where five fit), or than the clusters need to be there all at once (16 of 8 are not
    // at one CTA an SM: 40 x 512 x 8192 ran in two rounds), which is asked once a device.
    static std::atomic<int> at_once[qgi::MAX_DEVICES][9][17];
    int64_t each = (l.grid + ctx.num_sms - 1) / ctx.num_sms;
    for (;; ++each) {
        cfg.dynamicSmemBytes = std::max(G::smem(l.splits), std::min(MOST, uint32_t(SM_SMEM / each) / 1024 * 1024 - 1024));
        if (l.splits == 1 || each > 16 || cfg.dynamicSmemBytes == G::smem(l.splits)) break;
        std::atomic<int> &known = at_once[ctx.device][l.splits][each];
        int clusters = known.load(std::memory_order_relaxed);
        if (clusters == 0) {
            if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess) {
                cudaGetLastError();              // not kept: the even share will do, and the launch says what is wrong
                break;
            }
            clusters = std::max(clusters, 1);
            known.store(clusters, std::memory_order_relaxed);
        }
        if (int64_t(clusters) * l.splits >= l.grid) break;
    }
    return cudaLaunchKernelEx(&cfg, kern, tmW, tmX, a, l.splits, ctx.epi, ctx.err, ctx.timeout_ns);
}

// The block height that is estimated fastest (48 rows on 28672 x 8192, 64 on 8192 x 28672, 32 on 4096 x 4096).
template <int NH>
cudaError_t launch_tokens(const qgi::W8A8Args &a, const qgi::LaunchCtx &ctx, bool *encode_ok) {
    const Layout l2 = layout<Cfg<NH, 2, 8>>(a, ctx.num_sms), l3 = layout<Cfg<NH, 3, 6>>(a, ctx.num_sms),
                 l4 = layout<Cfg<NH, 4, 5>>(a, ctx.num_sms);
    if (l4.us <= l3.us && l4.us <= l2.us) return launch_nh<NH, 4, 5>(a, l4, ctx, encode_ok);
    return l3.us <= l2.us ? launch_nh<NH, 3, 6>(a, l3, ctx, encode_ok) : launch_nh<NH, 2, 8>(a, l2, ctx, encode_ok);
}

}  // namespace

namespace qgi {

cudaError_t launch_w8a8_decode(const W8A8Args &a, const LaunchCtx &ctx, bool *encode_ok) {
    if (a.M <= 8) return launch_tokens<1>(a, ctx, encode_ok);
    if (a.M <= 16) return launch_tokens<2>(a, ctx, encode_ok);
    if (a.M <= 32) return launch_nh<4, 2, 6>(a, layout<Cfg<4, 2, 6>>(a, ctx.num_sms), ctx, encode_ok);
    // past 32 tokens two fragments a block and four stages: sums take as many registers as 64 tokens need
    return launch_nh<8, 2, 4>(a, layout<Cfg<8, 2, 4>>(a, ctx.num_sms), ctx, encode_ok);
}

}  // namespace qgi

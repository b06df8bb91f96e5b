// kv_api.cu -- C ABI of the decode-serving operators: rotary frequencies, the paged key-value cache
// view, append, single-token attention and page operations.  Argument validation only; the kernels
// live in rope_append.cu, paged_attention.cu and kv_pages.cu.
#include <cmath>
#include <new>

#include "kv_index.h"
#include "kv_internal.h"

using qgi::fail;

namespace {

constexpr int64_t MAX_COUNT = (int64_t(1) << 31) - 1;
constexpr int64_t MAX_PAGES = int64_t(1) << 30;

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

qgemm_status cuda_fail(cudaError_t e, const char *what) {
    return fail(QGEMM_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Whether rows of `inner` bytes at these strides, over these extents, are disjoint: taken from the
// smallest stride up, each must step over all that the ones before it span.  *extent receives the
// bytes from the base to the end of the last row (-1 on overflow).
bool disjoint_rows(const int64_t (&n)[4], const int64_t *st, int64_t inner, int64_t *extent) {
    int order[4] = {0, 1, 2, 3};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (st[order[j]] < st[order[i]]) {
                const int t = order[i];
                order[i] = order[j];
                order[j] = t;
            }
    int64_t span = inner;
    *extent = -1;
    for (int i = 0; i < 4; ++i) {
        const int d = order[i];
        if (n[d] <= 1) continue;
        if (st[d] < span) return false;
        if (st[d] > (int64_t(1) << 62) / n[d]) return true;      // extent stays -1
        span += st[d] * (n[d] - 1);
        if (span > (int64_t(1) << 62)) return true;
    }
    *extent = span;
    return true;
}

qgemm_status check_16bit(int32_t dt, const char *what) {
    if (dt != QGEMM_F16 && dt != QGEMM_BF16)
        return fail(QGEMM_ERR_UNSUPPORTED_DTYPE, "%s: activations are F16 or BF16 (got %d)", what, dt);
    return QGEMM_OK;
}

// Rows [T, heads, d] of 16-bit elements at strides in elements: non-negative, 2-byte aligned.
qgemm_status check_rows(const void *x, int64_t ts, int64_t hs, const char *what) {
    if (!x) return fail(QGEMM_ERR_INVALID_ARG, "%s is NULL", what);
    if (ts < 0 || hs < 0) return fail(QGEMM_ERR_INVALID_ARG, "%s: negative stride", what);
    if (!aligned(x, 2)) return fail(QGEMM_ERR_MISALIGNED, "%s must be 2-byte aligned", what);
    return QGEMM_OK;
}

// The stride of a dimension of one is never stepped and may be anything.
void drop_unstepped(int64_t T, int64_t H, int64_t *ts, int64_t *hs) {
    if (T == 1) *ts = 0;
    if (H == 1) *hs = 0;
}

// An output's rows must not overlap, tokens outside heads or heads outside tokens.
qgemm_status check_output_rows(int64_t T, int64_t H, int64_t d, int64_t ts, int64_t hs, const char *what) {
    const int64_t n[4] = {T, H, 1, 1}, st[4] = {ts, hs, 0, 0};
    int64_t extent;
    if (!disjoint_rows(n, st, d, &extent))
        return fail(QGEMM_ERR_INVALID_ARG, "%s: rows overlap (strides %lld, %lld)", what, (long long)ts,
                    (long long)hs);
    return QGEMM_OK;
}

// A page table on the device: [max_seqs, max_pages] int32.
qgemm_status check_table(const qgemm_kv_cache *kv, const int32_t *table, int64_t stride, int64_t max_seqs,
                         int64_t max_pages) {
    if (max_seqs < 0 || max_pages < 0) return fail(QGEMM_ERR_INVALID_ARG, "negative page-table shape");
    // kernels step through a row's entries in 32 bits, 1024 at a time
    if (max_seqs > MAX_COUNT || max_pages > MAX_PAGES || max_pages > MAX_COUNT / kv->page_size)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE,
                    "page table of %lld x %lld pages of %lld tokens: a row holds fewer than 2^31 tokens in at most 2^30 pages",
                    (long long)max_seqs, (long long)max_pages, (long long)kv->page_size);
    if (max_seqs > 0 && max_pages > 0 && !table) return fail(QGEMM_ERR_INVALID_ARG, "page table is NULL");
    if (max_seqs > 1 && stride < max_pages)
        return fail(QGEMM_ERR_INVALID_ARG, "page-table stride %lld < %lld entries", (long long)stride,
                    (long long)max_pages);
    if (!aligned(table, 4)) return fail(QGEMM_ERR_MISALIGNED, "page table must be 4-byte aligned");
    return QGEMM_OK;
}

qgemm_status check_ints(const int32_t *p, const char *what) {
    if (!p) return fail(QGEMM_ERR_INVALID_ARG, "%s is NULL", what);
    if (!aligned(p, 4)) return fail(QGEMM_ERR_MISALIGNED, "%s must be 4-byte aligned", what);
    return QGEMM_OK;
}

}  // namespace

#define QG_TRY(expr)                                \
    do {                                            \
        const qgemm_status st_ = (expr);            \
        if (st_ != QGEMM_OK) return st_;            \
    } while (0)

extern "C" {

qgemm_status qgemm_create_rope(qgemm_rotation **out, int64_t rot_dim, int32_t interleaved, double base,
                               int32_t scaling, double factor, double original_len, double low_turns,
                               double high_turns, double mscale) {
    if (!out) return fail(QGEMM_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (rot_dim < 2 || rot_dim % 2) return fail(QGEMM_ERR_INVALID_ARG, "rot_dim must be even and >= 2 (got %lld)",
                                                (long long)rot_dim);
    if (rot_dim > 256) return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "rot_dim %lld > 256", (long long)rot_dim);
    if (interleaved != 0 && interleaved != 1)
        return fail(QGEMM_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if (!(base > 0) || !std::isfinite(base)) return fail(QGEMM_ERR_INVALID_ARG, "base must be finite and > 0");
    if (!std::isfinite((float)mscale)) return fail(QGEMM_ERR_INVALID_ARG, "mscale must be finite in fp32");
    if (scaling < QGEMM_ROPE_PLAIN || scaling > QGEMM_ROPE_BY_PARTS)
        return fail(QGEMM_ERR_INVALID_ARG, "unknown scaling %d", scaling);
    if (scaling != QGEMM_ROPE_PLAIN && (!(factor > 0) || !std::isfinite(factor)))
        return fail(QGEMM_ERR_INVALID_ARG, "factor must be finite and > 0");
    if (scaling == QGEMM_ROPE_BY_PARTS &&
        (!(original_len > 0) || !std::isfinite(original_len) || !std::isfinite(low_turns) ||
         !std::isfinite(high_turns) || !(high_turns > low_turns)))
        return fail(QGEMM_ERR_INVALID_ARG, "by parts: original_len > 0 and high_turns > low_turns");
    qgemm_rotation *r = new (std::nothrow) qgemm_rotation();
    if (!r) return fail(QGEMM_ERR_INVALID_ARG, "out of host memory");
    r->rot_dim = (int32_t)rot_dim;
    r->interleaved = interleaved;
    r->mscale = (float)mscale;
    const double two_pi = 6.283185307179586476925286766559;
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        double w = std::pow(base, -2.0 * (double)i / (double)rot_dim);
        if (scaling == QGEMM_ROPE_LINEAR) w /= factor;
        if (scaling == QGEMM_ROPE_BY_PARTS) {
            double keep = (original_len * w / two_pi - low_turns) / (high_turns - low_turns);
            keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
            w *= keep + (1 - keep) / factor;
        }
        if (!std::isfinite(w)) {
            delete r;
            return fail(QGEMM_ERR_INVALID_ARG, "the frequency of pair %lld is not finite", (long long)i);
        }
        // the fraction of a turn as 64 bits; whole turns of a position do not show
        const double turn = w / two_pi, frac = turn - std::floor(turn);
        const double scaled = std::ldexp(frac, 64);
        r->freq[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
    }
    *out = r;
    return QGEMM_OK;
}

void qgemm_destroy_rope(qgemm_rotation *rope) { delete rope; }

qgemm_status qgemm_create_kv_cache(qgemm_kv_cache **out, int32_t dtype, int64_t layers, int64_t pages,
                                   int64_t heads, int64_t page_size, int64_t d, void *k, void *v,
                                   const int64_t *strides, uint8_t *k_scales, uint8_t *v_scales,
                                   const int64_t *scale_strides) {
    if (!out) return fail(QGEMM_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (dtype != QGEMM_F16 && dtype != QGEMM_BF16 && dtype != QGEMM_E4M3)
        return fail(QGEMM_ERR_UNSUPPORTED_DTYPE, "a cache is F16, BF16 or E4M3 (got %d)", dtype);
    if (layers < 1 || pages < 1 || heads < 1 || page_size < 1)
        return fail(QGEMM_ERR_INVALID_ARG, "layers, pages, heads and page_size must be >= 1");
    if (d != 64 && d != 128)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "head dimension must be 64 or 128 (got %lld)", (long long)d);
    if (layers > 65536 || pages > MAX_PAGES || heads > 65536 || page_size > 65536)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "layers, heads, page_size <= 65536, pages <= 2^30");
    if (layers * heads * page_size >= (int64_t(1) << 31))
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "a page has 2^31 rows or more in all layers");
    if (!k || !v || !strides) return fail(QGEMM_ERR_INVALID_ARG, "k, v or strides is NULL");
    if (k == v) return fail(QGEMM_ERR_INVALID_ARG, "k and v are the same plane");
    const bool e4m3 = dtype == QGEMM_E4M3;
    if (e4m3 && (!k_scales || !v_scales || !scale_strides))
        return fail(QGEMM_ERR_INVALID_ARG, "an E4M3 cache needs scale planes and their strides");
    if (e4m3 && k_scales == v_scales) return fail(QGEMM_ERR_INVALID_ARG, "k_scales and v_scales are the same plane");
    if (!e4m3 && (k_scales || v_scales)) return fail(QGEMM_ERR_UNSUPPORTED_DTYPE, "only E4M3 takes scale planes");
    const int64_t n[4] = {layers, pages, heads, page_size};
    int64_t st[4] = {0, 0, 0, 0}, sst[4] = {0, 0, 0, 0}, extent = 0, sextent = 0;
    for (int i = 0; i < 4; ++i) {
        if (n[i] > 1) {
            st[i] = strides[i];
            if (st[i] < 0) return fail(QGEMM_ERR_INVALID_ARG, "negative stride");
            if (st[i] % 16) return fail(QGEMM_ERR_MISALIGNED, "strides must be multiples of 16 bytes");
            if (e4m3) {
                sst[i] = scale_strides[i];
                if (sst[i] < 0) return fail(QGEMM_ERR_INVALID_ARG, "negative scale stride");
                if (sst[i] % 4) return fail(QGEMM_ERR_MISALIGNED, "scale strides must be multiples of 4 bytes");
            }
        }
    }
    if (!aligned(k, 16) || !aligned(v, 16)) return fail(QGEMM_ERR_MISALIGNED, "k and v must be 16-byte aligned");
    if (e4m3 && (!aligned(k_scales, 4) || !aligned(v_scales, 4)))
        return fail(QGEMM_ERR_MISALIGNED, "scale planes must be 4-byte aligned");
    if (!disjoint_rows(n, st, e4m3 ? d : 2 * d, &extent))
        return fail(QGEMM_ERR_INVALID_ARG, "the strides make rows overlap");
    if (e4m3 && !disjoint_rows(n, sst, 4, &sextent))
        return fail(QGEMM_ERR_INVALID_ARG, "the scale strides make rows of 4 bytes overlap");
    if (extent < 0 || sextent < 0) return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "cache larger than 2^62 bytes");
    qgemm_kv_cache *c = new (std::nothrow) qgemm_kv_cache();
    if (!c) return fail(QGEMM_ERR_INVALID_ARG, "out of host memory");
    c->dtype = dtype;
    c->layers = layers;
    c->pages = pages;
    c->heads = heads;
    c->page_size = page_size;
    c->d = d;
    c->k = static_cast<uint8_t *>(k);
    c->v = static_cast<uint8_t *>(v);
    c->ks = k_scales;
    c->vs = v_scales;
    for (int i = 0; i < 4; ++i) {
        c->st[i] = st[i];
        c->sst[i] = sst[i];
    }
    // a token stride that is never stepped still tells the page copy its rows are dense
    if (page_size == 1) c->st[3] = e4m3 ? d : 2 * d;
    c->extent = extent;
    c->sextent = sextent;
    auto unit_of = [&](const int64_t *s, int64_t least, int64_t *unit) {
        int64_t bits = least << 16, last = 0;            // at most 2^16 of the least
        for (int i = 1; i < 4; ++i) {
            bits |= s[i];
            last += (n[i] - 1) * s[i];
        }
        *unit = bits & -bits;
        return last / *unit < (int64_t(1) << 32);
    };
    c->near = unit_of(st, 16, &c->unit);
    c->near = unit_of(sst, 4, &c->sunit) && c->near;
    *out = c;
    return QGEMM_OK;
}

void qgemm_destroy_kv_cache(qgemm_kv_cache *kv) { delete kv; }

qgemm_status qgemm_rope(const void *X, int64_t x_token_stride, int64_t x_head_stride, void *Y,
                        int64_t y_token_stride, int64_t y_head_stride, int32_t dtype, int64_t T, int64_t heads,
                        int64_t d, const int32_t *positions, const qgemm_rotation *rope, int32_t inverse,
                        void *stream) {
    QG_TRY(check_16bit(dtype, "qgemm_rope"));
    if (!rope) return fail(QGEMM_ERR_INVALID_ARG, "rope is NULL");
    if (T < 0 || heads < 0 || d < 0) return fail(QGEMM_ERR_INVALID_ARG, "negative shape");
    if (inverse != 0 && inverse != 1) return fail(QGEMM_ERR_INVALID_ARG, "inverse must be 0 or 1");
    if (d > 256 || d < rope->rot_dim)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "head dimension must be in rot_dim (%d) .. 256 (got %lld)",
                    rope->rot_dim, (long long)d);
    if (T > MAX_COUNT || heads > 65536)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "tokens < 2^31, heads <= 65536");
    if (T == 0 || heads == 0) return QGEMM_OK;
    drop_unstepped(T, heads, &x_token_stride, &x_head_stride);
    drop_unstepped(T, heads, &y_token_stride, &y_head_stride);
    QG_TRY(check_rows(X, x_token_stride, x_head_stride, "X"));
    QG_TRY(check_rows(Y, y_token_stride, y_head_stride, "Y"));
    QG_TRY(check_output_rows(T, heads, d, y_token_stride, y_head_stride, "Y"));
    QG_TRY(check_ints(positions, "positions"));
    qgi::AppendArgs a = {};
    a.T = (int32_t)T;
    a.d = (int32_t)d;
    a.bf16 = dtype == QGEMM_BF16;
    a.q = {X, Y, x_token_stride, x_head_stride, y_token_stride, y_head_stride, (int32_t)heads};
    a.pos = positions;
    a.rope = rope;
    a.inverse = inverse;
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    const cudaError_t e = qgi::launch_rope_append(a, ctx);
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_rope launch");
}

qgemm_status qgemm_kv_append(const qgemm_kv_cache *kv, int64_t layer, const void *K, int64_t k_token_stride,
                             int64_t k_head_stride, const void *V, int64_t v_token_stride, int64_t v_head_stride,
                             int32_t dtype, int64_t T, const int32_t *seqs, const int32_t *positions,
                             const int32_t *page_table, int64_t table_stride, int64_t max_seqs, int64_t max_pages,
                             const qgemm_rotation *rope, const void *Q, int64_t q_token_stride,
                             int64_t q_head_stride, int64_t q_heads, void *Q_out, int64_t qo_token_stride,
                             int64_t qo_head_stride, void *stream) {
    if (!kv) return fail(QGEMM_ERR_INVALID_ARG, "cache is NULL");
    QG_TRY(check_16bit(dtype, "qgemm_kv_append"));
    if (kv->dtype != QGEMM_E4M3 && kv->dtype != dtype)
        return fail(QGEMM_ERR_UNSUPPORTED_DTYPE, "a 16-bit cache takes activations of its own type");
    if (layer < 0 || layer >= kv->layers)
        return fail(QGEMM_ERR_INVALID_ARG, "layer %lld of %lld", (long long)layer, (long long)kv->layers);
    if (T < 0 || q_heads < 0) return fail(QGEMM_ERR_INVALID_ARG, "negative shape");
    if (T > MAX_COUNT || q_heads > 65536)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "tokens < 2^31, heads <= 65536");
    if (rope && rope->rot_dim > kv->d)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "rot_dim %d > head dimension %lld", rope->rot_dim, (long long)kv->d);
    QG_TRY(check_table(kv, page_table, table_stride, max_seqs, max_pages));
    if (T == 0) return QGEMM_OK;
    drop_unstepped(T, kv->heads, &k_token_stride, &k_head_stride);
    drop_unstepped(T, kv->heads, &v_token_stride, &v_head_stride);
    drop_unstepped(T, q_heads, &q_token_stride, &q_head_stride);
    drop_unstepped(T, q_heads, &qo_token_stride, &qo_head_stride);
    QG_TRY(check_rows(K, k_token_stride, k_head_stride, "K"));
    QG_TRY(check_rows(V, v_token_stride, v_head_stride, "V"));
    QG_TRY(check_ints(seqs, "seqs"));
    QG_TRY(check_ints(positions, "positions"));
    qgi::AppendArgs a = {};
    if (q_heads > 0) {
        QG_TRY(check_rows(Q, q_token_stride, q_head_stride, "Q"));
        QG_TRY(check_rows(Q_out, qo_token_stride, qo_head_stride, "Q_out"));
        QG_TRY(check_output_rows(T, q_heads, kv->d, qo_token_stride, qo_head_stride, "Q_out"));
        a.q = {Q, Q_out, q_token_stride, q_head_stride, qo_token_stride, qo_head_stride, (int32_t)q_heads};
    }
    a.T = (int32_t)T;
    a.d = (int32_t)kv->d;
    a.bf16 = dtype == QGEMM_BF16;
    a.k = K;
    a.kt = k_token_stride;
    a.kh = k_head_stride;
    a.v = V;
    a.vt = v_token_stride;
    a.vh = v_head_stride;
    a.kv = kv;
    a.layer = layer;
    a.seqs = seqs;
    a.pos = positions;
    a.table = page_table;
    a.table_stride = table_stride;
    a.max_seqs = (int32_t)max_seqs;
    a.max_pages = (int32_t)max_pages;
    a.rope = rope;
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    const cudaError_t e = qgi::launch_rope_append(a, ctx);
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_kv_append launch");
}

qgemm_status qgemm_paged_attention_workspace_bytes(const qgemm_kv_cache *kv, int64_t batch, int64_t q_heads,
                                                   int64_t *bytes) {
    if (!kv || !bytes) return fail(QGEMM_ERR_INVALID_ARG, "cache or bytes is NULL");
    if (batch < 0 || q_heads < 1 || q_heads % kv->heads)
        return fail(QGEMM_ERR_INVALID_ARG, "q_heads must be a multiple of the cache's %lld heads",
                    (long long)kv->heads);
    if (batch > 65536 || q_heads > 65536)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "batch and q_heads <= 65536");
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(nullptr, &ctx));
    *bytes = (int64_t)qgi::paged_attention_workspace(kv, ctx.num_sms);
    return QGEMM_OK;
}

qgemm_status qgemm_paged_attention(const void *Q, int64_t q_batch_stride, int64_t q_head_stride, int32_t dtype,
                                   int64_t batch, int64_t q_heads, const qgemm_kv_cache *kv, int64_t layer,
                                   const int32_t *page_table, int64_t table_stride, int64_t max_seqs,
                                   int64_t max_pages, const int32_t *lens, const int32_t *seqs, void *O,
                                   int64_t o_batch_stride, int64_t o_head_stride, float *lse, float scale,
                                   int64_t window, void *workspace, int64_t workspace_bytes, void *stream) {
    if (!kv) return fail(QGEMM_ERR_INVALID_ARG, "cache is NULL");
    QG_TRY(check_16bit(dtype, "qgemm_paged_attention"));
    if (kv->dtype != QGEMM_E4M3 && kv->dtype != dtype)
        return fail(QGEMM_ERR_UNSUPPORTED_DTYPE, "queries on a 16-bit cache have its type");
    if (layer < 0 || layer >= kv->layers)
        return fail(QGEMM_ERR_INVALID_ARG, "layer %lld of %lld", (long long)layer, (long long)kv->layers);
    if (batch < 0 || q_heads < 1 || q_heads % kv->heads)
        return fail(QGEMM_ERR_INVALID_ARG, "q_heads must be a multiple of the cache's %lld heads",
                    (long long)kv->heads);
    if (batch > 65536 || q_heads > 65536)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "batch and q_heads <= 65536");
    if (!std::isfinite(scale) || !(scale > 0))
        return fail(QGEMM_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (window < 0) return fail(QGEMM_ERR_INVALID_ARG, "negative window");
    QG_TRY(check_table(kv, page_table, table_stride, max_seqs, max_pages));
    if (batch == 0) return QGEMM_OK;
    drop_unstepped(batch, q_heads, &q_batch_stride, &q_head_stride);
    drop_unstepped(batch, q_heads, &o_batch_stride, &o_head_stride);
    QG_TRY(check_rows(Q, q_batch_stride, q_head_stride, "Q"));
    QG_TRY(check_rows(O, o_batch_stride, o_head_stride, "O"));
    if (!aligned(Q, 16) || !aligned(O, 16) || q_batch_stride % 8 || q_head_stride % 8 || o_batch_stride % 8 ||
        o_head_stride % 8)
        return fail(QGEMM_ERR_MISALIGNED, "Q and O must be 16-byte aligned with strides in multiples of 8");
    QG_TRY(check_output_rows(batch, q_heads, kv->d, o_batch_stride, o_head_stride, "O"));
    if (max_seqs < 1) return fail(QGEMM_ERR_INVALID_ARG, "the page table has no rows");
    if (!seqs && batch > max_seqs)
        return fail(QGEMM_ERR_INVALID_ARG, "batch %lld > %lld page-table rows", (long long)batch,
                    (long long)max_seqs);
    if (!kv->near)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "a layer's rows lie 2^32 units (%lld bytes of rows, %lld of scales) apart",
                    (long long)kv->unit, (long long)kv->sunit);
    QG_TRY(check_ints(lens, "lens"));
    if (!aligned(seqs, 4) || !aligned(lse, 4)) return fail(QGEMM_ERR_MISALIGNED, "seqs and lse must be 4-byte aligned");
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    if (batch * q_heads * (max_pages * kv->page_size / 128 + 3) / ctx.num_sms > MAX_COUNT)
        return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "more than 2^31 tiles of 128 tokens an SM");
    const int64_t need = (int64_t)qgi::paged_attention_workspace(kv, ctx.num_sms);
    if (!workspace || workspace_bytes < need)
        return fail(QGEMM_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed",
                    (long long)(workspace ? workspace_bytes : 0), (long long)need);
    if (!aligned(workspace, 16)) return fail(QGEMM_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    qgi::PagedAttnArgs a = {};
    a.q = Q;
    a.qb = q_batch_stride;
    a.qh = q_head_stride;
    a.o = O;
    a.ob = o_batch_stride;
    a.oh = o_head_stride;
    a.lse = lse;
    a.bf16 = dtype == QGEMM_BF16;
    a.B = (int32_t)batch;
    a.hq = (int32_t)q_heads;
    a.kv = kv;
    a.layer = layer;
    a.table = page_table;
    a.lens = lens;
    a.seqs = seqs;
    a.table_stride = table_stride;
    a.max_seqs = (int32_t)max_seqs;
    a.max_pages = (int32_t)max_pages;
    a.window = (int32_t)(window > MAX_COUNT ? MAX_COUNT : window);
    a.scale = scale;
    a.workspace = workspace;
    const cudaError_t e = qgi::launch_paged_attention(a, ctx);
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_paged_attention launch");
}

// The table, lengths and counts of a page operation, checked and gathered.
static qgemm_status page_args(qgi::PageArgs *a, const qgemm_kv_cache *kv, int32_t *page_table, int64_t table_stride,
                              int64_t max_seqs, int64_t max_pages, int32_t *lens, int32_t *refs) {
    if (!kv) return fail(QGEMM_ERR_INVALID_ARG, "cache is NULL");
    QG_TRY(check_table(kv, page_table, table_stride, max_seqs, max_pages));
    if (max_seqs < 1 || max_pages < 1) return fail(QGEMM_ERR_INVALID_ARG, "the page table is empty");
    QG_TRY(check_ints(lens, "lens"));
    QG_TRY(check_ints(refs, "refs"));
    a->kv = kv;
    a->table = page_table;
    a->table_stride = table_stride;
    a->max_seqs = (int32_t)max_seqs;
    a->max_pages = (int32_t)max_pages;
    a->lens = lens;
    a->refs = refs;
    return QGEMM_OK;
}

static qgemm_status check_items(int64_t n) {
    if (n < 0) return fail(QGEMM_ERR_INVALID_ARG, "negative count");
    if (n > (1 << 24)) return fail(QGEMM_ERR_UNSUPPORTED_SHAPE, "more than 2^24 items");
    return QGEMM_OK;
}

qgemm_status qgemm_kv_resize(const qgemm_kv_cache *kv, int32_t *page_table, int64_t table_stride, int64_t max_seqs,
                             int64_t max_pages, int32_t *lens, int32_t *refs, const int32_t *seqs,
                             const int32_t *new_lens, int64_t n, void *stream) {
    qgi::PageArgs a = {};
    QG_TRY(page_args(&a, kv, page_table, table_stride, max_seqs, max_pages, lens, refs));
    QG_TRY(check_items(n));
    if (n == 0) return QGEMM_OK;
    QG_TRY(check_ints(seqs, "seqs"));
    if (!aligned(new_lens, 4)) return fail(QGEMM_ERR_MISALIGNED, "new_lens must be 4-byte aligned");
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    const cudaError_t e = qgi::launch_kv_resize(a, seqs, new_lens, (int32_t)n, ctx);
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_kv_resize");
}

qgemm_status qgemm_kv_fork(const qgemm_kv_cache *kv, int32_t *page_table, int64_t table_stride, int64_t max_seqs,
                           int64_t max_pages, int32_t *lens, int32_t *refs, const int32_t *parents,
                           const int32_t *children, int64_t n, void *stream) {
    qgi::PageArgs a = {};
    QG_TRY(page_args(&a, kv, page_table, table_stride, max_seqs, max_pages, lens, refs));
    QG_TRY(check_items(n));
    if (n == 0) return QGEMM_OK;
    QG_TRY(check_ints(parents, "parents"));
    QG_TRY(check_ints(children, "children"));
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    const cudaError_t e = qgi::launch_kv_fork(a, parents, children, (int32_t)n, ctx);
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_kv_fork");
}

qgemm_status qgemm_kv_compact(const qgemm_kv_cache *kv, int32_t *page_table, int64_t table_stride, int64_t max_seqs,
                              int64_t max_pages, int32_t *lens, int32_t *refs, void *stream) {
    qgi::PageArgs a = {};
    QG_TRY(page_args(&a, kv, page_table, table_stride, max_seqs, max_pages, lens, refs));
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    const cudaError_t e = qgi::launch_kv_compact(a, ctx);
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_kv_compact");
}

qgemm_status qgemm_kv_copy_pages(const qgemm_kv_cache *kv, const int32_t *src, const int32_t *dst, int64_t n,
                                 void *stream) {
    if (!kv) return fail(QGEMM_ERR_INVALID_ARG, "cache is NULL");
    QG_TRY(check_items(n));
    if (n == 0) return QGEMM_OK;
    QG_TRY(check_ints(src, "src"));
    QG_TRY(check_ints(dst, "dst"));
    qgi::LaunchCtx ctx;
    QG_TRY(qgi::launch_ctx(stream, &ctx));
    const cudaError_t e = qgi::launch_kv_copy_pages(kv, src, dst, (int32_t)n, ctx);
    return e == cudaSuccess ? QGEMM_OK : cuda_fail(e, "qgemm_kv_copy_pages");
}

}  // extern "C"

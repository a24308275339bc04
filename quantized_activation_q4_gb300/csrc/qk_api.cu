// libqk C ABI: argument checks on the host, then the kernel launchers.
//
// Every check happens before anything is enqueued, so a bad call leaves the
// stream untouched (minfer doc 52 "r49 A-quantize prepass shared-A dedup",
// section 3.1: errors surface at entry, not as a fault in a later launch).
// Aliasing outputs are refused (llama.cpp PR #117 "activation image
// emission", Coverage: unsafe input/output aliases keep the original path).

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "qk_internal.cuh"
#include "qk_kv.cuh"

namespace qk {

static thread_local char g_err[512] = "";
static std::atomic<uint64_t> g_launches{0};

qk_status fail(qk_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}

qk_status check_launch(const char *what) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return QK_OK;
}

void count_launch(unsigned n) { g_launches.fetch_add(n, std::memory_order_relaxed); }

}  // namespace qk

using namespace qk;

#define REQUIRE(cond, status, ...) \
    do {                           \
        if (!(cond)) return fail(status, __VA_ARGS__); \
    } while (0)

constexpr int QK_W_LAST = QK_W_Q4_G128;
// Largest N and K of the group-scaled weights and of the routed prefill: indices of whole units past them fit an int.
constexpr int64_t MOST_NK = INT32_MAX - 1023;

static bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static qk_status check_proj_common(int32_t wtype, const void *w, int64_t N, int64_t K, int64_t img_row_blocks) {
    REQUIRE(wtype >= QK_W_Q4_0 && wtype <= QK_W_LAST, QK_ERR_ARG, "bad wtype %d", (int)wtype);
    REQUIRE(w, QK_ERR_ARG, "null weight pointer");
    REQUIRE(aligned(w, 16), QK_ERR_ARG, "packed weights must be 16-byte aligned");
    const int64_t most = group_scaled(wtype) ? MOST_NK : INT32_MAX;
    REQUIRE(N >= 1 && N <= most && K >= 32 && K <= most, QK_ERR_ARG, "N or K out of range");
    REQUIRE(K % group_size(wtype) == 0, QK_ERR_SHAPE, "K=%lld is not a multiple of %d", (long long)K,
            group_size(wtype));
    REQUIRE(K / QB <= img_row_blocks, QK_ERR_SHAPE, "K=%lld reaches past the image row (%lld blocks)",
            (long long)K, (long long)img_row_blocks);
    return QK_OK;
}

// No output lies over any projection's weights: CTAs read the one while others write the other.
template <typename YSpan, typename WSpan>
static qk_status outputs_off_weights(int32_t n_proj, YSpan y_of, WSpan w_of) {
    for (int j = 0; j < n_proj; j++)
        for (int i = 0; i < n_proj; i++)
            REQUIRE(!overlap(y_of(j), w_of(i)), QK_ERR_ALIAS, "y of projection %d overlaps the weights of projection %d", j, i);
    return QK_OK;
}

namespace qk {
// Every check of qk_mmvq except those of the workspace: the image, T, the
// projections, their outputs and aliasing between them.
qk_status mmvq_validate(const void *img, int64_t img_row_blocks, int64_t T, int32_t n_proj, const qk_proj *projs) {
    REQUIRE(img && projs, QK_ERR_ARG, "null pointer");
    REQUIRE(aligned(img, 4), QK_ERR_ARG, "img not 4-byte aligned");
    REQUIRE(T >= 1 && img_row_blocks >= 1, QK_ERR_ARG, "T or img_row_blocks < 1");
    REQUIRE(T <= 8, QK_ERR_UNSUPPORTED, "T=%lld > 8 (use qk_mmq for larger batches)", (long long)T);
    REQUIRE(n_proj >= 1 && n_proj <= 8, QK_ERR_UNSUPPORTED, "n_proj=%d not in 1..8", (int)n_proj);
    Span si = span(img, (size_t)(T * img_row_blocks * Q8_1_BYTES));
    for (int j = 0; j < n_proj; j++) {
        const qk_proj &p = projs[j];
        qk_status st = check_proj_common(p.wtype, p.w, p.N, p.K, img_row_blocks);
        if (st != QK_OK) return st;
        REQUIRE(p.y && aligned(p.y, 4), QK_ERR_ARG, "projection %d: y is null or misaligned", j);
        REQUIRE(p.y_stride >= p.N, QK_ERR_SHAPE, "projection %d: y_stride < N", j);
        Span sy = span(p.y, rows_span(T, p.y_stride * 4, p.N * 4));
        REQUIRE(!overlap(sy, si), QK_ERR_ALIAS, "projection %d: y overlaps img", j);
        for (int i = 0; i < j; i++) {
            REQUIRE(!rows_overlap(projs[i].y, projs[i].y_stride * 4, projs[i].N * 4, p.y, p.y_stride * 4, p.N * 4, T),
                    QK_ERR_ALIAS, "outputs of projections %d and %d overlap", i, j);
        }
    }
    return outputs_off_weights(
        n_proj, [&](int j) { return span(projs[j].y, rows_span(T, projs[j].y_stride * 4, projs[j].N * 4)); },
        [&](int j) { return span(projs[j].w, (size_t)packed_bytes(projs[j].wtype, projs[j].N, projs[j].K)); });
}
}  // namespace qk

extern "C" {

const char *qk_status_string(qk_status s) {
    switch (s) {
        case QK_OK: return "QK_OK";
        case QK_ERR_ARG: return "QK_ERR_ARG";
        case QK_ERR_SHAPE: return "QK_ERR_SHAPE";
        case QK_ERR_ALIAS: return "QK_ERR_ALIAS";
        case QK_ERR_WORKSPACE: return "QK_ERR_WORKSPACE";
        case QK_ERR_UNSUPPORTED: return "QK_ERR_UNSUPPORTED";
        case QK_ERR_CUDA: return "QK_ERR_CUDA";
    }
    return "QK_ERR_UNKNOWN";
}

const char *qk_last_error(void) { return g_err; }
const char *qk_last_error_string(void) { return g_err; }

uint64_t qk_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

// ------------------------------------------------------------------ image
static qk_status check_quant_in(const float *x, int64_t T, int64_t K, int64_t x_stride) {
    REQUIRE(T >= 0 && T <= INT32_MAX, QK_ERR_ARG, "T=%lld out of range", (long long)T);
    REQUIRE(K >= 1 && K <= (1LL << 25), QK_ERR_ARG, "K=%lld out of range", (long long)K);
    REQUIRE(x || T == 0, QK_ERR_ARG, "x is null");
    REQUIRE(x_stride >= K, QK_ERR_SHAPE, "x_stride=%lld < K=%lld", (long long)x_stride, (long long)K);
    REQUIRE(aligned(x, 4), QK_ERR_ARG, "x not 4-byte aligned");
    return QK_OK;
}

qk_status qk_quantize_q8_1(const float *x, int64_t T, int64_t K, int64_t x_stride, void *img,
                           int64_t img_row_blocks, const int32_t *d_live_rows, qk_stream stream) {
    qk_status st = check_quant_in(x, T, K, x_stride);
    if (st != QK_OK) return st;
    REQUIRE(img || T == 0, QK_ERR_ARG, "img is null");
    REQUIRE(aligned(img, 4), QK_ERR_ARG, "img not 4-byte aligned");
    REQUIRE(img_row_blocks >= ceil_div(K, QB), QK_ERR_SHAPE, "img_row_blocks=%lld < ceil(K/32)=%lld",
            (long long)img_row_blocks, (long long)ceil_div(K, QB));
    REQUIRE(img_row_blocks <= (1 << 20), QK_ERR_ARG, "img_row_blocks > 2^20");
    Span sx = span(x, rows_span(T, x_stride * 4, K * 4));
    Span si = span(img, (size_t)(T * img_row_blocks * Q8_1_BYTES));
    REQUIRE(!overlap(sx, si), QK_ERR_ALIAS, "img overlaps x");
    return launch_quantize_q8_1(x, (int)T, (int)K, x_stride, static_cast<uint8_t *>(img), img_row_blocks,
                                d_live_rows, (cudaStream_t)stream);
}

qk_status qk_quantize_q8_0(const float *x, int64_t T, int64_t K, int64_t x_stride, int8_t *qs,
                           uint16_t *d, int64_t row_blocks, const int32_t *d_live_rows, qk_stream stream) {
    qk_status st = check_quant_in(x, T, K, x_stride);
    if (st != QK_OK) return st;
    REQUIRE((qs && d) || T == 0, QK_ERR_ARG, "qs or d is null");
    REQUIRE(aligned(qs, 4) && aligned(d, 2), QK_ERR_ARG, "qs must be 4-byte and d 2-byte aligned");
    REQUIRE(row_blocks >= ceil_div(K, QB), QK_ERR_SHAPE, "row_blocks=%lld < ceil(K/32)", (long long)row_blocks);
    REQUIRE(row_blocks <= (1 << 20), QK_ERR_ARG, "row_blocks > 2^20");
    Span sx = span(x, rows_span(T, x_stride * 4, K * 4));
    Span sq = span(qs, (size_t)(T * row_blocks * QB));
    Span sd = span(d, (size_t)(T * row_blocks * 2));
    REQUIRE(!overlap(sx, sq) && !overlap(sx, sd) && !overlap(sq, sd), QK_ERR_ALIAS, "qs/d overlap x or each other");
    return launch_quantize_q8_0(x, (int)T, (int)K, x_stride, qs, d, row_blocks, d_live_rows, (cudaStream_t)stream);
}

// ------------------------------------------------------------------ image memo
void qk_image_memo_clear(qk_image_memo *memo) {
    if (memo) *memo = qk_image_memo{};
}

int32_t qk_image_memo_match(const qk_image_memo *m, int32_t format, const float *x, int64_t T, int64_t K,
                            int64_t x_stride, const void *dst0, const void *dst1, int64_t row_blocks,
                            qk_stream stream) {
    return m && m->format != QK_MEMO_EMPTY && m->format == format && m->x == x && m->T == T && m->K == K &&
           m->x_stride == x_stride && m->row_blocks == row_blocks && m->dst0 == dst0 && m->dst1 == dst1 &&
           m->stream == stream;
}

static qk_status memo_record(qk_image_memo *m, qk_status st, int32_t format, const float *x, int64_t T,
                             int64_t K, int64_t x_stride, const void *dst0, const void *dst1, int64_t row_blocks,
                             qk_stream stream) {
    qk_image_memo_clear(m);
    if (st == QK_OK) {
        m->format = format;
        m->x = x;
        m->T = T;
        m->K = K;
        m->x_stride = x_stride;
        m->row_blocks = row_blocks;
        m->dst0 = dst0;
        m->dst1 = dst1;
        m->stream = stream;
    }
    return st;
}

qk_status qk_image_memo_quantize_q8_0(qk_image_memo *memo, const float *x, int64_t T, int64_t K, int64_t x_stride,
                                      int8_t *qs, uint16_t *d, int64_t row_blocks, int32_t *hit, qk_stream stream) {
    REQUIRE(memo, QK_ERR_ARG, "memo is null");
    if (!hit) {
        qk_image_memo_clear(memo);
        return fail(QK_ERR_ARG, "hit is null");
    }
    *hit = qk_image_memo_match(memo, QK_MEMO_Q8_0, x, T, K, x_stride, qs, d, row_blocks, stream);
    if (*hit) return QK_OK;
    const qk_status st = qk_quantize_q8_0(x, T, K, x_stride, qs, d, row_blocks, nullptr, stream);
    return memo_record(memo, st, QK_MEMO_Q8_0, x, T, K, x_stride, qs, d, row_blocks, stream);
}

qk_status qk_image_memo_quantize_q8_1(qk_image_memo *memo, const float *x, int64_t T, int64_t K, int64_t x_stride,
                                      void *img, int64_t img_row_blocks, int32_t *hit, qk_stream stream) {
    REQUIRE(memo, QK_ERR_ARG, "memo is null");
    if (!hit) {
        qk_image_memo_clear(memo);
        return fail(QK_ERR_ARG, "hit is null");
    }
    *hit = qk_image_memo_match(memo, QK_MEMO_Q8_1, x, T, K, x_stride, img, nullptr, img_row_blocks, stream);
    if (*hit) return QK_OK;
    const qk_status st = qk_quantize_q8_1(x, T, K, x_stride, img, img_row_blocks, nullptr, stream);
    return memo_record(memo, st, QK_MEMO_Q8_1, x, T, K, x_stride, img, nullptr, img_row_blocks, stream);
}

// ------------------------------------------------------------------ producers
qk_status qk_rmsnorm_q8_1(const float *x, int64_t T, int64_t K, int64_t x_stride, qk_norm_kind kind,
                          const float *w, const float *b, float scale, float eps, float *y,
                          int64_t y_stride, void *img, int64_t img_row_blocks,
                          const int32_t *d_live_rows, qk_stream stream) {
    qk_status st = check_quant_in(x, T, K, x_stride);
    if (st != QK_OK) return st;
    REQUIRE(kind >= QK_NORM_PLAIN && kind <= QK_NORM_SCALE, QK_ERR_ARG, "bad norm kind %d", (int)kind);
    REQUIRE(K % QB == 0, QK_ERR_SHAPE, "K=%lld is not a whole number of 32-blocks", (long long)K);
    REQUIRE(K <= 32768, QK_ERR_UNSUPPORTED, "K=%lld > 32768 (a row is kept in registers)", (long long)K);
    REQUIRE((y && img) || T == 0, QK_ERR_ARG, "y or img is null");
    const bool need_w = kind == QK_NORM_MUL || kind == QK_NORM_MUL_ADD;
    REQUIRE(!need_w || w, QK_ERR_ARG, "w is null for a MUL kind");
    REQUIRE(kind != QK_NORM_MUL_ADD || b, QK_ERR_ARG, "b is null for MUL_ADD");
    REQUIRE(y_stride >= K, QK_ERR_SHAPE, "y_stride < K");
    REQUIRE(img_row_blocks >= K / QB, QK_ERR_SHAPE, "img_row_blocks < K/32");
    REQUIRE(aligned(y, 4) && aligned(img, 4) && aligned(w, 4) && aligned(b, 4), QK_ERR_ARG, "misaligned pointer");
    Span sx = span(x, rows_span(T, x_stride * 4, K * 4));
    Span sy = span(y, rows_span(T, y_stride * 4, K * 4));
    Span si = span(img, (size_t)(T * img_row_blocks * Q8_1_BYTES));
    Span sw = span(need_w ? w : nullptr, need_w ? (size_t)K * 4 : 0);
    Span sb = span(kind == QK_NORM_MUL_ADD ? b : nullptr, kind == QK_NORM_MUL_ADD ? (size_t)K * 4 : 0);
    REQUIRE(!overlap(sy, sx) && !overlap(sy, si) && !overlap(si, sx) && !overlap(sy, sw) && !overlap(sy, sb) &&
                !overlap(si, sw) && !overlap(si, sb),
            QK_ERR_ALIAS, "y or img overlaps an input or each other");
    return launch_rmsnorm_q8_1(x, (int)T, (int)K, x_stride, (int)kind, w, b, scale, eps, y, y_stride,
                               static_cast<uint8_t *>(img), img_row_blocks, d_live_rows, (cudaStream_t)stream);
}

qk_status qk_rmsnorm_q8_0(const float *x, int64_t T, int64_t K, int64_t x_stride, qk_norm_kind kind,
                          const float *w, const float *b, float scale, float eps, float *y, int64_t y_stride,
                          int8_t *qs, uint16_t *d, int64_t row_blocks, const int32_t *d_live_rows,
                          qk_stream stream) {
    qk_status st = check_quant_in(x, T, K, x_stride);
    if (st != QK_OK) return st;
    REQUIRE(kind >= QK_NORM_PLAIN && kind <= QK_NORM_SCALE, QK_ERR_ARG, "bad norm kind %d", (int)kind);
    REQUIRE(K % QB == 0, QK_ERR_SHAPE, "K=%lld is not a whole number of 32-blocks", (long long)K);
    REQUIRE(K <= 32768, QK_ERR_UNSUPPORTED, "K=%lld > 32768 (a row is kept in registers)", (long long)K);
    REQUIRE((y && qs && d) || T == 0, QK_ERR_ARG, "y, qs or d is null");
    const bool need_w = kind == QK_NORM_MUL || kind == QK_NORM_MUL_ADD;
    REQUIRE(!need_w || w, QK_ERR_ARG, "w is null for a MUL kind");
    REQUIRE(kind != QK_NORM_MUL_ADD || b, QK_ERR_ARG, "b is null for MUL_ADD");
    REQUIRE(y_stride >= K, QK_ERR_SHAPE, "y_stride < K");
    REQUIRE(row_blocks >= K / QB, QK_ERR_SHAPE, "row_blocks < K/32");
    REQUIRE(aligned(y, 4) && aligned(qs, 16) && aligned(d, 4) && aligned(w, 4) && aligned(b, 4), QK_ERR_ARG,
            "misaligned pointer (qs must be 16-byte aligned)");
    Span sx = span(x, rows_span(T, x_stride * 4, K * 4));
    Span sy = span(y, rows_span(T, y_stride * 4, K * 4));
    Span sq = span(qs, (size_t)(T * row_blocks * QB)), sd = span(d, (size_t)(T * row_blocks * 2));
    Span sw = span(need_w ? w : nullptr, need_w ? (size_t)K * 4 : 0);
    Span sb = span(kind == QK_NORM_MUL_ADD ? b : nullptr, kind == QK_NORM_MUL_ADD ? (size_t)K * 4 : 0);
    const Span outs[3] = {sy, sq, sd}, ins[3] = {sx, sw, sb};
    for (int o = 0; o < 3; o++) {
        for (int i = 0; i < 3; i++) REQUIRE(!overlap(outs[o], ins[i]), QK_ERR_ALIAS, "an output overlaps an input");
        for (int q = 0; q < o; q++) REQUIRE(!overlap(outs[o], outs[q]), QK_ERR_ALIAS, "outputs overlap each other");
    }
    return launch_rmsnorm_q8_0(x, (int)T, (int)K, x_stride, (int)kind, w, b, scale, eps, y, y_stride, qs, d,
                               row_blocks, d_live_rows, (cudaStream_t)stream);
}

qk_status qk_glu_q8_1(qk_glu_kind kind, qk_glu_layout layout, const float *a, int64_t a_stride,
                      const float *b, int64_t b_stride, int64_t T, int64_t N, float *out,
                      int64_t out_stride, void *img, int64_t img_row_blocks, const int32_t *d_live_rows,
                      qk_stream stream) {
    return qk_glu_q8_1_ex(kind, layout, a, a_stride, b, b_stride, T, N, out, out_stride, img, img_row_blocks,
                          1.702f, 7.0f, d_live_rows, stream);
}

qk_status qk_glu_q8_1_ex(qk_glu_kind kind, qk_glu_layout layout, const float *a, int64_t a_stride,
                         const float *b, int64_t b_stride, int64_t T, int64_t N, float *out,
                         int64_t out_stride, void *img, int64_t img_row_blocks, float alpha, float limit,
                         const int32_t *d_live_rows, qk_stream stream) {
    REQUIRE(kind >= QK_GLU_SWIGLU && kind <= QK_GLU_SWIGLU_CLAMP, QK_ERR_ARG, "bad glu kind %d", (int)kind);
    REQUIRE(std::isfinite(alpha) && std::isfinite(limit) && limit > 0.0f, QK_ERR_ARG,
            "alpha must be finite and limit positive and finite");
    REQUIRE(layout >= QK_GLU_SEPARATE && layout <= QK_GLU_PACKED_SWAPPED, QK_ERR_ARG, "bad glu layout %d", (int)layout);
    REQUIRE(T >= 0 && T <= INT32_MAX && N >= 1 && N <= (1LL << 25), QK_ERR_ARG, "T or N out of range");
    REQUIRE(N % QB == 0, QK_ERR_SHAPE, "N=%lld is not a whole number of 32-blocks", (long long)N);
    REQUIRE((a && out && img && (layout != QK_GLU_SEPARATE || b)) || T == 0, QK_ERR_ARG, "null pointer");
    const int64_t a_row = layout == QK_GLU_SEPARATE ? N : 2 * N;
    REQUIRE(a_stride >= a_row, QK_ERR_SHAPE, "a_stride too small");
    REQUIRE(layout != QK_GLU_SEPARATE || b_stride >= N, QK_ERR_SHAPE, "b_stride < N");
    REQUIRE(out_stride >= N && img_row_blocks >= N / QB, QK_ERR_SHAPE, "out_stride or img_row_blocks too small");
    REQUIRE(aligned(a, 4) && aligned(b, 4) && aligned(out, 4) && aligned(img, 4), QK_ERR_ARG, "misaligned pointer");
    Span sa = span(a, rows_span(T, a_stride * 4, a_row * 4));
    Span sb = span(layout == QK_GLU_SEPARATE ? b : nullptr,
                   layout == QK_GLU_SEPARATE ? rows_span(T, b_stride * 4, N * 4) : 0);
    Span so = span(out, rows_span(T, out_stride * 4, N * 4));
    Span si = span(img, (size_t)(T * img_row_blocks * Q8_1_BYTES));
    REQUIRE(!overlap(so, sa) && !overlap(so, sb) && !overlap(so, si) && !overlap(si, sa) && !overlap(si, sb),
            QK_ERR_ALIAS, "out or img overlaps an input or each other");
    return launch_glu_q8_1((int)kind, (int)layout, a, a_stride, b, b_stride, (int)T, (int)N, out, out_stride,
                           static_cast<uint8_t *>(img), img_row_blocks, alpha, limit, d_live_rows,
                           (cudaStream_t)stream);
}

qk_status qk_glu_q8_0(qk_glu_kind kind, qk_glu_layout layout, qk_elem elem, const void *a, int64_t a_stride,
                      const void *b, int64_t b_stride, int64_t T, int64_t N, float *out, int64_t out_stride,
                      int8_t *qs, uint16_t *d, int64_t row_blocks, float alpha, float limit,
                      const int32_t *d_live_rows, qk_stream stream) {
    REQUIRE(kind >= QK_GLU_SWIGLU && kind <= QK_GLU_SWIGLU_CLAMP, QK_ERR_ARG, "bad glu kind %d", (int)kind);
    REQUIRE(std::isfinite(alpha) && std::isfinite(limit) && limit > 0.0f, QK_ERR_ARG,
            "alpha must be finite and limit positive and finite");
    REQUIRE(layout >= QK_GLU_SEPARATE && layout <= QK_GLU_PACKED_SWAPPED, QK_ERR_ARG, "bad glu layout %d", (int)layout);
    REQUIRE(elem == QK_ELEM_F32 || elem == QK_ELEM_BF16, QK_ERR_ARG, "bad element type %d", (int)elem);
    REQUIRE(T >= 0 && T <= INT32_MAX && N >= 1 && N <= (1LL << 25), QK_ERR_ARG, "T or N out of range");
    REQUIRE(N % QB == 0, QK_ERR_SHAPE, "N=%lld is not a whole number of 32-blocks", (long long)N);
    const bool separate = layout == QK_GLU_SEPARATE;
    REQUIRE((a && qs && d && (!separate || b)) || T == 0, QK_ERR_ARG, "null pointer");
    const int64_t es = elem == QK_ELEM_F32 ? 4 : 2, a_row = separate ? N : 2 * N;
    REQUIRE(a_stride >= a_row, QK_ERR_SHAPE, "a_stride too small");
    REQUIRE(!separate || b_stride >= N, QK_ERR_SHAPE, "b_stride < N");
    REQUIRE((!out || out_stride >= N) && row_blocks >= N / QB, QK_ERR_SHAPE, "out_stride or row_blocks too small");
    REQUIRE(row_blocks <= (1 << 20), QK_ERR_ARG, "row_blocks > 2^20");
    REQUIRE(aligned(a, es) && (!separate || aligned(b, es)) && aligned(out, 4) && aligned(qs, 4) && aligned(d, 2),
            QK_ERR_ARG, "misaligned pointer");
    Span sa = span(a, rows_span(T, a_stride * es, a_row * es));
    Span sb = span(separate ? b : nullptr, separate ? rows_span(T, b_stride * es, N * es) : 0);
    Span so = span(out, out ? rows_span(T, out_stride * 4, N * 4) : 0);
    Span sq = span(qs, (size_t)(T * row_blocks * QB)), sd = span(d, (size_t)(T * row_blocks * 2));
    const Span outs[3] = {so, sq, sd};
    for (int o = 0; o < 3; o++) {
        REQUIRE(!overlap(outs[o], sa) && !overlap(outs[o], sb), QK_ERR_ALIAS, "an output overlaps an input");
        for (int q = 0; q < o; q++) REQUIRE(!overlap(outs[o], outs[q]), QK_ERR_ALIAS, "outputs overlap each other");
    }
    return launch_glu_q8_0((int)kind, (int)layout, (int)elem, a, a_stride, b, b_stride, (int)T, (int)N, out, out_stride,
                           qs, d, row_blocks, alpha, limit, d_live_rows, (cudaStream_t)stream);
}

// ------------------------------------------------------------------ weights
size_t qk_weight_packed_bytes(qk_wtype wtype, int64_t N, int64_t K) {
    if (wtype < QK_W_Q4_0 || (int)wtype > QK_W_LAST || N < 0 || K < 0) return 0;
    return (size_t)packed_bytes(wtype, N, K);
}

qk_status qk_weight_pack(qk_wtype wtype, const void *blocks, int64_t N, int64_t K, void *packed,
                         size_t packed_bytes_, qk_stream stream) {
    REQUIRE(wtype >= QK_W_Q4_0 && (int)wtype <= QK_W_LAST, QK_ERR_ARG, "bad wtype %d", (int)wtype);
    const int64_t most = group_scaled(wtype) ? MOST_NK : INT32_MAX;
    REQUIRE(N >= 1 && K >= 32 && N <= most && K <= most, QK_ERR_ARG, "N or K out of range");
    const int G = group_size(wtype);
    REQUIRE(K % G == 0, QK_ERR_SHAPE, "K=%lld is not a multiple of %d", (long long)K, G);
    REQUIRE(blocks && packed, QK_ERR_ARG, "null pointer");
    REQUIRE(aligned(packed, 16), QK_ERR_ARG, "packed must be 16-byte aligned");
    const size_t need = (size_t)packed_bytes(wtype, N, K);
    REQUIRE(packed_bytes_ >= need, QK_ERR_WORKSPACE, "packed_bytes=%zu < %zu", packed_bytes_, need);
    const int64_t block = wtype == QK_W_Q4_0 ? Q4_0_BYTES : wtype == QK_W_Q8_0 ? Q8_0_BYTES : 4 + G / 2;
    const size_t src = (size_t)(N * (K / G) * block);
    REQUIRE(!overlap(span(blocks, src), span(packed, need)), QK_ERR_ALIAS, "packed overlaps blocks");
    if (group_scaled(wtype))
        return launch_weight_pack_g(wtype, static_cast<const uint8_t *>(blocks), N, K,
                                    static_cast<uint8_t *>(packed), (cudaStream_t)stream);
    return launch_weight_pack(wtype, static_cast<const uint8_t *>(blocks), N, K, static_cast<uint8_t *>(packed),
                              (cudaStream_t)stream);
}

// ------------------------------------------------------------------ projections

size_t qk_mmvq_workspace_bytes(int32_t n_proj, const qk_proj *projs) {
    if (n_proj < 1 || n_proj > 8 || !projs) return 0;
    size_t need = 0;
    for (int wt = QK_W_Q4_0; wt <= QK_W_Q8_0; wt++) {
        qk_proj group[8];
        int n = 0;
        for (int j = 0; j < n_proj; j++)
            if (projs[j].wtype == wt) group[n++] = projs[j];
        if (n == 0) continue;
        const size_t g = (size_t)mmvq_workspace_bytes(n, group);
        need = g > need ? g : need;
    }
    return need;
}

qk_status qk_device_faults(uint32_t *faults) {
    REQUIRE(faults, QK_ERR_ARG, "faults is null");
    uint32_t a = 0, b = 0, c = 0, d = 0, e = 0, f = 0, g = 0;
    qk_status st = read_device_faults(&a);
    if (st == QK_OK) st = read_mmq_faults(&b);
    if (st == QK_OK) st = read_mmq_id_faults(&c);
    if (st == QK_OK) st = read_mmvq_g_faults(&d);
    if (st == QK_OK) st = read_attn_decode_faults(&e);
    if (st == QK_OK) st = read_attn_prefill_faults(&f);
    if (st == QK_OK) st = read_attn_wide_faults(&g);
    *faults = a | b | c | d | e | f | g;
    return st;
}

qk_status qk_selftest_wait_timeout(qk_stream stream) { return launch_wait_selftest((cudaStream_t)stream); }

qk_status qk_mmvq(const void *img, int64_t img_row_blocks, int64_t T, int32_t n_proj, const qk_proj *projs,
                  const int32_t *d_live_rows, void *ws, size_t ws_bytes, qk_stream stream) {
    qk_status vs = mmvq_validate(img, img_row_blocks, T, n_proj, projs);
    if (vs != QK_OK) return vs;
    Span si = span(img, (size_t)(T * img_row_blocks * Q8_1_BYTES));
    bool need_ws = false;
    for (int j = 0; j < n_proj; j++) need_ws |= !group_scaled(projs[j].wtype);
    REQUIRE(!need_ws || (ws && aligned(ws, 16)), QK_ERR_WORKSPACE, "workspace null or not 16-byte aligned");
    // one launch per weight type present, in order on the stream; they share ws
    for (int wt = QK_W_Q4_0; wt <= QK_W_Q8_0; wt++) {
        qk_proj group[8];
        int n = 0;
        for (int j = 0; j < n_proj; j++)
            if (projs[j].wtype == wt) group[n++] = projs[j];
        if (n == 0) continue;
        const size_t need = (size_t)mmvq_workspace_bytes(n, group);
        REQUIRE(ws_bytes >= need, QK_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
        Span sws = span(ws, need);
        REQUIRE(!overlap(sws, si), QK_ERR_ALIAS, "workspace overlaps img");
        for (int j = 0; j < n_proj; j++)
            REQUIRE(!overlap(sws, span(projs[j].y, rows_span(T, projs[j].y_stride * 4, projs[j].N * 4))) &&
                        !overlap(sws, span(projs[j].w, (size_t)packed_bytes(projs[j].wtype, projs[j].N, projs[j].K))),
                    QK_ERR_ALIAS, "workspace overlaps projection %d", j);
    }
    for (int wt = QK_W_Q4_0; wt <= QK_W_Q8_0; wt++) {
        qk_proj group[8];
        int n = 0;
        for (int j = 0; j < n_proj; j++)
            if (projs[j].wtype == wt) group[n++] = projs[j];
        if (n == 0) continue;
        qk_status st = launch_mmvq(static_cast<const uint8_t *>(img), img_row_blocks, (int)T, n, group,
                                   d_live_rows, ws, ws_bytes, (cudaStream_t)stream);
        if (st != QK_OK) return st;
    }
    for (int wt = QK_W_Q4_G64; wt <= QK_W_Q4_G128; wt++) {
        qk_proj group[8];
        int n = 0;
        for (int j = 0; j < n_proj; j++)
            if (projs[j].wtype == wt) group[n++] = projs[j];
        if (n == 0) continue;
        qk_status st = launch_mmvq_g(static_cast<const uint8_t *>(img), img_row_blocks, (int)T, n, group, d_live_rows,
                                     (cudaStream_t)stream);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

static qk_status mmvq_id_common(const void *img, int64_t img_row_blocks, int64_t rows, int32_t k, int32_t n_proj,
                                const qk_proj_id *projs, const int32_t *counts, const int32_t *offsets,
                                const int32_t *items, bool per_pair, qk_stream stream) {
    REQUIRE(img && projs && counts && offsets && items, QK_ERR_ARG, "null pointer");
    REQUIRE(aligned(img, 4), QK_ERR_ARG, "img not 4-byte aligned");
    REQUIRE(aligned(counts, 4) && aligned(offsets, 4) && aligned(items, 4), QK_ERR_ARG, "misaligned plan pointer");
    REQUIRE(rows >= 1 && rows <= (1 << 24) && k >= 1 && k <= 64 && img_row_blocks >= 1, QK_ERR_ARG,
            "rows, k or img_row_blocks out of range");
    REQUIRE(n_proj >= 1 && n_proj <= 8, QK_ERR_UNSUPPORTED, "n_proj=%d not in 1..8", (int)n_proj);
    Span si = span(img, (size_t)((per_pair ? rows * k : rows) * img_row_blocks * Q8_1_BYTES));
    // the plan is read while outputs are written: no output may overlap it
    const int64_t E = projs[0].n_experts;
    const Span plan[3] = {span(counts, (size_t)(E > 0 ? E : 0) * 4), span(offsets, (size_t)(E > 0 ? E + 1 : 0) * 4),
                          span(items, (size_t)(rows * k * 4))};
    for (int j = 0; j < n_proj; j++) {
        const qk_proj_id &p = projs[j];
        qk_status st = check_proj_common(p.wtype, p.w, p.N, p.K, img_row_blocks);
        if (st != QK_OK) return st;
        REQUIRE(p.n_experts >= 1 && p.n_experts <= 1024, QK_ERR_UNSUPPORTED, "n_experts=%d", (int)p.n_experts);
        REQUIRE(p.y && aligned(p.y, 4), QK_ERR_ARG, "projection %d: y is null or misaligned", j);
        REQUIRE(projs[0].n_experts == p.n_experts, QK_ERR_ARG, "projections disagree on n_experts");
        Span sy = span(p.y, (size_t)(rows * k * p.N * 4));
        REQUIRE(!overlap(sy, si), QK_ERR_ALIAS, "projection %d: y overlaps img", j);
        REQUIRE(!overlap(sy, plan[0]) && !overlap(sy, plan[1]) && !overlap(sy, plan[2]), QK_ERR_ALIAS,
                "projection %d: y overlaps counts, offsets or items", j);
        for (int i = 0; i < j; i++)
            REQUIRE(!overlap(sy, span(projs[i].y, (size_t)(rows * k * projs[i].N * 4))), QK_ERR_ALIAS,
                    "outputs of projections %d and %d overlap", i, j);
    }
    const qk_status alias = outputs_off_weights(
        n_proj, [&](int j) { return span(projs[j].y, (size_t)(rows * k * projs[j].N * 4)); },
        [&](int j) { return span(projs[j].w, (size_t)packed_bytes(projs[j].wtype, projs[j].N, projs[j].K) * E); });
    if (alias != QK_OK) return alias;
    // the routed kernels count their work items in int: (passes of any plan) x (row tiles or strips) < 2^31
    int64_t tiles = 0;
    for (int j = 0; j < n_proj; j++) tiles += ceil_div(projs[j].N, group_scaled(projs[j].wtype) ? STRIP_ROWS : UNIT_ROWS);
    REQUIRE(((rows * k + 7) / 8 + E) * tiles < (1LL << 31), QK_ERR_UNSUPPORTED,
            "rows * k * row tiles too large for one routed launch");
    for (int wt = QK_W_Q4_0; wt <= QK_W_LAST; wt++) {
        qk_proj_id group[8];
        int n = 0;
        for (int j = 0; j < n_proj; j++)
            if (projs[j].wtype == wt) group[n++] = projs[j];
        if (n == 0) continue;
        qk_status st = (group_scaled(wt) ? launch_mmvq_g_id : launch_mmvq_id)(
            static_cast<const uint8_t *>(img), img_row_blocks, (int)rows, k, n, group, counts, offsets, items, per_pair,
            (cudaStream_t)stream);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

qk_status qk_mmvq_id(const void *img, int64_t img_row_blocks, int64_t rows, int32_t k, int32_t n_proj,
                     const qk_proj_id *projs, const int32_t *counts, const int32_t *offsets,
                     const int32_t *items, qk_stream stream) {
    return mmvq_id_common(img, img_row_blocks, rows, k, n_proj, projs, counts, offsets, items, false, stream);
}

qk_status qk_mmvq_id_slots(const void *img, int64_t img_row_blocks, int64_t rows, int32_t k, int32_t n_proj,
                           const qk_proj_id *projs, const int32_t *counts, const int32_t *offsets,
                           const int32_t *items, qk_stream stream) {
    return mmvq_id_common(img, img_row_blocks, rows, k, n_proj, projs, counts, offsets, items, true, stream);
}

qk_status qk_moe_combine(const float *expert_out, int64_t out_stride, const float *wts, int64_t rows, int32_t k,
                         int64_t N, float *y, int64_t y_stride, const int32_t *d_live_rows, qk_stream stream) {
    REQUIRE(expert_out && wts && y, QK_ERR_ARG, "null pointer");
    REQUIRE(rows >= 0 && rows <= (1 << 24) && k >= 1 && k <= 64 && N >= 1 && N <= (1LL << 25), QK_ERR_ARG,
            "rows, k or N out of range");
    REQUIRE(out_stride >= N && y_stride >= N, QK_ERR_SHAPE, "out_stride or y_stride < N");
    REQUIRE(aligned(expert_out, 16) && aligned(y, 16) && out_stride % 4 == 0 && y_stride % 4 == 0 && N % 4 == 0,
            QK_ERR_ARG, "expert_out and y must be 16-byte aligned with strides and N multiples of 4");
    Span se = span(expert_out, rows_span(rows * k, out_stride * 4, N * 4));
    Span sw = span(wts, (size_t)(rows * k * 4));
    Span sy = span(y, rows_span(rows, y_stride * 4, N * 4));
    REQUIRE(!overlap(sy, se) && !overlap(sy, sw), QK_ERR_ALIAS, "y overlaps expert_out or wts");
    if (rows == 0) return QK_OK;
    return launch_moe_combine(expert_out, out_stride, wts, (int)rows, k, (int)N, y, y_stride, d_live_rows,
                              (cudaStream_t)stream);
}

qk_status qk_moe_combine_bf16(const uint16_t *expert_out, int64_t out_stride, const float *wts, int64_t rows,
                              int32_t k, int64_t N, float *y, int64_t y_stride, const int32_t *d_live_rows,
                              qk_stream stream) {
    REQUIRE(expert_out && wts && y, QK_ERR_ARG, "null pointer");
    REQUIRE(rows >= 0 && rows <= (1 << 24) && k >= 1 && k <= 64 && N >= 1 && N <= (1LL << 25), QK_ERR_ARG,
            "rows, k or N out of range");
    REQUIRE(out_stride >= N && y_stride >= N, QK_ERR_SHAPE, "out_stride or y_stride < N");
    REQUIRE(aligned(expert_out, 8) && aligned(wts, 4) && aligned(y, 16) && out_stride % 4 == 0 && y_stride % 4 == 0 &&
                N % 4 == 0,
            QK_ERR_ARG, "expert_out must be 8-byte and y 16-byte aligned with strides and N multiples of 4");
    Span se = span(expert_out, rows_span(rows * k, out_stride * 2, N * 2));
    Span sw = span(wts, (size_t)(rows * k * 4));
    Span sy = span(y, rows_span(rows, y_stride * 4, N * 4));
    REQUIRE(!overlap(sy, se) && !overlap(sy, sw), QK_ERR_ALIAS, "y overlaps expert_out or wts");
    if (rows == 0) return QK_OK;
    return launch_moe_combine_bf16(expert_out, out_stride, wts, (int)rows, k, (int)N, y, y_stride, d_live_rows,
                                   (cudaStream_t)stream);
}

// ------------------------------------------------------------------ routing
qk_status qk_topk_route(const float *logits, int64_t rows, int32_t E, int32_t k, int32_t *ids, float *wts,
                        const int32_t *d_live_rows, qk_stream stream) {
    REQUIRE(logits && ids && wts, QK_ERR_ARG, "null pointer");
    REQUIRE(rows >= 0 && rows <= (1 << 24) && E >= 1 && k >= 1, QK_ERR_ARG, "rows, E or k out of range");
    REQUIRE(E <= 256 && k <= 32 && k <= E, QK_ERR_UNSUPPORTED, "E=%d k=%d (need E <= 256, k <= min(32, E))", E, k);
    Span sl = span(logits, (size_t)(rows * E * 4));
    Span si = span(ids, (size_t)(rows * k * 4));
    Span sw = span(wts, (size_t)(rows * k * 4));
    REQUIRE(!overlap(si, sl) && !overlap(sw, sl) && !overlap(si, sw), QK_ERR_ALIAS, "ids/wts overlap logits or each other");
    return launch_topk_route(logits, (int)rows, E, k, ids, wts, d_live_rows, (cudaStream_t)stream);
}

qk_status qk_moe_plan(const int32_t *ids, int64_t rows, int32_t k, int32_t E, int32_t *counts, int32_t *offsets,
                      int32_t *items, const int32_t *d_live_rows, qk_stream stream) {
    REQUIRE(ids && counts && offsets && items, QK_ERR_ARG, "null pointer");
    REQUIRE(rows >= 0 && rows <= (1 << 24) && k >= 1 && k <= 64 && E >= 1, QK_ERR_ARG, "rows, k or E out of range");
    REQUIRE(E <= 1024, QK_ERR_UNSUPPORTED, "E=%d > 1024", E);
    Span s_ids = span(ids, (size_t)(rows * k * 4));
    Span sc = span(counts, (size_t)E * 4), so = span(offsets, (size_t)(E + 1) * 4);
    Span sit = span(items, (size_t)(rows * k * 4));
    REQUIRE(!overlap(sc, s_ids) && !overlap(so, s_ids) && !overlap(sit, s_ids) && !overlap(sc, so) &&
                !overlap(sc, sit) && !overlap(so, sit),
            QK_ERR_ALIAS, "plan outputs overlap ids or each other");
    return launch_moe_plan(ids, (int)rows, k, E, counts, offsets, items, d_live_rows, (cudaStream_t)stream);
}

qk_status qk_route_plan(const float *logits, int64_t rows, int32_t E, int32_t k, int32_t *ids, float *wts,
                        int32_t *counts, int32_t *offsets, int32_t *items, const int32_t *d_live_rows,
                        qk_stream stream) {
    REQUIRE(logits && ids && wts && counts && offsets && items, QK_ERR_ARG, "null pointer");
    REQUIRE(rows >= 0 && rows <= (1 << 24) && E >= 1 && k >= 1, QK_ERR_ARG, "rows, E or k out of range");
    REQUIRE(E <= 256 && k <= 32 && k <= E, QK_ERR_UNSUPPORTED, "E=%d k=%d (need E <= 256, k <= min(32, E))", E, k);
    Span sl = span(logits, (size_t)(rows * E * 4));
    Span si = span(ids, (size_t)(rows * k * 4));
    Span sw = span(wts, (size_t)(rows * k * 4));
    Span sc = span(counts, (size_t)E * 4), so = span(offsets, (size_t)(E + 1) * 4);
    Span sit = span(items, (size_t)(rows * k * 4));
    const Span outs[5] = {si, sw, sc, so, sit};
    for (int a = 0; a < 5; a++) {
        REQUIRE(!overlap(outs[a], sl), QK_ERR_ALIAS, "an output overlaps logits");
        for (int b = 0; b < a; b++) REQUIRE(!overlap(outs[a], outs[b]), QK_ERR_ALIAS, "outputs overlap each other");
    }
    // rows == 0 still launches: like qk_moe_plan, the plan of no pairs writes zero counts and offsets
    return launch_route_plan(logits, (int)rows, E, k, ids, wts, counts, offsets, items, d_live_rows,
                             (cudaStream_t)stream);
}

// ------------------------------------------------------------------ prefill
size_t qk_mmq_workspace_bytes(int64_t T, int32_t n_proj, const qk_proj *projs) {
    if (T < 1 || n_proj < 1 || n_proj > 8 || !projs) return 0;
    int64_t kmax = 0;
    for (int j = 0; j < n_proj; j++) kmax = projs[j].K > kmax ? projs[j].K : kmax;
    return (size_t)mmq_workspace_bytes(T, kmax);
}

qk_status qk_mmq(const int8_t *qs, const uint16_t *d, int64_t row_blocks, int64_t T, int32_t n_proj,
                 const qk_proj *projs, void *ws, size_t ws_bytes, qk_stream stream) {
    REQUIRE(qs && d && projs, QK_ERR_ARG, "null pointer");
    REQUIRE(T >= 1 && T <= INT32_MAX && row_blocks >= 1, QK_ERR_ARG, "T or row_blocks out of range");
    REQUIRE(n_proj >= 1 && n_proj <= 8, QK_ERR_UNSUPPORTED, "n_proj=%d not in 1..8", (int)n_proj);
    REQUIRE(aligned(qs, 16) && aligned(d, 4), QK_ERR_ARG, "qs must be 16-byte and d 4-byte aligned");
    Span sq = span(qs, (size_t)(T * row_blocks * QB)), sd = span(d, (size_t)(T * row_blocks * 2));
    for (int j = 0; j < n_proj; j++) {
        const qk_proj &p = projs[j];
        qk_status st = check_proj_common(p.wtype, p.w, p.N, p.K, row_blocks);
        if (st != QK_OK) return st;
        REQUIRE(p.wtype == QK_W_Q4_0, QK_ERR_UNSUPPORTED, "qk_mmq takes Q4_0 weights");
        REQUIRE(p.y && p.y_stride >= p.N, QK_ERR_SHAPE, "projection %d: y null or y_stride < N", j);
        REQUIRE(aligned(p.y, 4), QK_ERR_ARG, "projection %d: y is misaligned", j);
        Span sy = span(p.y, rows_span(T, p.y_stride * 4, p.N * 4));
        REQUIRE(!overlap(sy, sq) && !overlap(sy, sd), QK_ERR_ALIAS, "projection %d: y overlaps the image", j);
        for (int i = 0; i < j; i++)
            REQUIRE(!rows_overlap(projs[i].y, projs[i].y_stride * 4, projs[i].N * 4, p.y, p.y_stride * 4, p.N * 4, T),
                    QK_ERR_ALIAS, "outputs of projections %d and %d overlap", i, j);
    }
    const qk_status alias = outputs_off_weights(
        n_proj, [&](int j) { return span(projs[j].y, rows_span(T, projs[j].y_stride * 4, projs[j].N * 4)); },
        [&](int j) { return span(projs[j].w, (size_t)packed_bytes(projs[j].wtype, projs[j].N, projs[j].K)); });
    if (alias != QK_OK) return alias;
    const size_t need = qk_mmq_workspace_bytes(T, n_proj, projs);
    REQUIRE(ws && aligned(ws, 128), QK_ERR_WORKSPACE, "workspace null or not 128-byte aligned");
    REQUIRE(ws_bytes >= need, QK_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    Span sws = span(ws, need);
    REQUIRE(!overlap(sws, sq) && !overlap(sws, sd), QK_ERR_ALIAS, "workspace overlaps the image");
    for (int j = 0; j < n_proj; j++)
        REQUIRE(!overlap(sws, span(projs[j].y, rows_span(T, projs[j].y_stride * 4, projs[j].N * 4))) &&
                    !overlap(sws, span(projs[j].w, (size_t)packed_bytes(projs[j].wtype, projs[j].N, projs[j].K))),
                QK_ERR_ALIAS, "workspace overlaps projection %d", j);
    return launch_mmq(qs, d, row_blocks, (int)T, n_proj, projs, ws, ws_bytes, (cudaStream_t)stream);
}

// ------------------------------------------------------------------ routed prefill
size_t qk_mmq_id_workspace_bytes(int64_t rows, int32_t k, int32_t n_proj, const qk_proj_id16 *projs) {
    if (rows < 1 || rows > (1 << 24) || k < 1 || k > 64 || n_proj < 1 || n_proj > 8 || !projs) return 0;
    int64_t kmax = 0;
    for (int j = 0; j < n_proj; j++) {
        if (projs[j].K < QB || projs[j].K > MOST_NK) return 0;
        kmax = projs[j].K > kmax ? projs[j].K : kmax;
    }
    return (size_t)mmq_id_workspace_bytes(rows * k, kmax);
}

static qk_status mmq_id_common(const int8_t *qs, const uint16_t *d, int64_t row_blocks, int64_t rows, int32_t k,
                               int32_t n_proj, const qk_proj_id16 *projs, const int32_t *counts,
                               const int32_t *offsets, const int32_t *items, void *ws, size_t ws_bytes, bool per_pair,
                               qk_stream stream) {
    REQUIRE(qs && d && projs && counts && offsets && items, QK_ERR_ARG, "null pointer");
    REQUIRE(rows >= 1 && rows <= (1 << 24) && k >= 1 && k <= 64 && row_blocks >= 1, QK_ERR_ARG,
            "rows, k or row_blocks out of range");
    REQUIRE(n_proj >= 1 && n_proj <= 8, QK_ERR_UNSUPPORTED, "n_proj=%d not in 1..8", (int)n_proj);
    REQUIRE(aligned(qs, 16) && aligned(d, 4), QK_ERR_ARG, "qs must be 16-byte and d 4-byte aligned");
    REQUIRE(aligned(counts, 4) && aligned(offsets, 4) && aligned(items, 4), QK_ERR_ARG, "misaligned plan pointer");
    const int64_t pairs = rows * k, img_rows = per_pair ? pairs : rows;
    const int64_t E = projs[0].n_experts;
    REQUIRE(E >= 1 && E <= 1024, QK_ERR_UNSUPPORTED, "n_experts=%lld", (long long)E);
    const Span sq = span(qs, (size_t)(img_rows * row_blocks * QB)), sd = span(d, (size_t)(img_rows * row_blocks * 2));
    const Span ins[5] = {sq, sd, span(counts, (size_t)E * 4), span(offsets, (size_t)(E + 1) * 4),
                         span(items, (size_t)(pairs * 4))};
    int64_t tiles = 0;
    for (int j = 0; j < n_proj; j++) {
        const qk_proj_id16 &p = projs[j];
        qk_status st = check_proj_common(p.wtype, p.w, p.N, p.K, row_blocks);
        if (st != QK_OK) return st;
        REQUIRE(p.wtype != QK_W_Q8_0, QK_ERR_UNSUPPORTED, "projection %d: Q8_0 weights are not taken", j);
        REQUIRE(p.N <= MOST_NK && p.K <= MOST_NK, QK_ERR_ARG, "projection %d: N or K out of range", j);
        REQUIRE(p.n_experts == E, QK_ERR_ARG, "projections disagree on n_experts");
        REQUIRE(p.y && aligned(p.y, 2), QK_ERR_ARG, "projection %d: y is null or misaligned", j);
        REQUIRE(p.y_stride >= p.N, QK_ERR_SHAPE, "projection %d: y_stride < N", j);
        const Span sy = span(p.y, rows_span(pairs, p.y_stride * 2, p.N * 2));
        for (int i = 0; i < 5; i++)
            REQUIRE(!overlap(sy, ins[i]), QK_ERR_ALIAS, "projection %d: y overlaps the image or the plan", j);
        for (int i = 0; i < j; i++)
            REQUIRE(!rows_overlap(projs[i].y, projs[i].y_stride * 2, projs[i].N * 2, p.y, p.y_stride * 2, p.N * 2, pairs),
                    QK_ERR_ALIAS, "outputs of projections %d and %d overlap", i, j);
        tiles += ceil_div(p.N, UNIT_ROWS);
    }
    const qk_status alias = outputs_off_weights(
        n_proj, [&](int j) { return span(projs[j].y, rows_span(pairs, projs[j].y_stride * 2, projs[j].N * 2)); },
        [&](int j) { return span(projs[j].w, (size_t)(packed_bytes(projs[j].wtype, projs[j].N, projs[j].K) * E)); });
    if (alias != QK_OK) return alias;
    // work items (passes of any plan x row tiles) are counted in int
    REQUIRE((pairs / 128 + E) * tiles < (1LL << 31), QK_ERR_UNSUPPORTED, "rows * k * row tiles too large for one launch");
    const size_t need = qk_mmq_id_workspace_bytes(rows, k, n_proj, projs);
    REQUIRE(ws && aligned(ws, 128), QK_ERR_WORKSPACE, "workspace null or not 128-byte aligned");
    REQUIRE(ws_bytes >= need, QK_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    const Span sws = span(ws, need);
    for (int i = 0; i < 5; i++) REQUIRE(!overlap(sws, ins[i]), QK_ERR_ALIAS, "workspace overlaps the image or the plan");
    for (int j = 0; j < n_proj; j++)
        REQUIRE(!overlap(sws, span(projs[j].y, rows_span(pairs, projs[j].y_stride * 2, projs[j].N * 2))) &&
                    !overlap(sws, span(projs[j].w, (size_t)(packed_bytes(projs[j].wtype, projs[j].N, projs[j].K) * E))),
                QK_ERR_ALIAS, "workspace overlaps projection %d", j);
    return launch_mmq_id(qs, d, row_blocks, (int)rows, k, n_proj, projs, counts, offsets, items, per_pair, ws,
                         (cudaStream_t)stream);
}

qk_status qk_mmq_id(const int8_t *qs, const uint16_t *d, int64_t row_blocks, int64_t rows, int32_t k, int32_t n_proj,
                    const qk_proj_id16 *projs, const int32_t *counts, const int32_t *offsets, const int32_t *items,
                    void *ws, size_t ws_bytes, qk_stream stream) {
    return mmq_id_common(qs, d, row_blocks, rows, k, n_proj, projs, counts, offsets, items, ws, ws_bytes, false, stream);
}

qk_status qk_mmq_id_slots(const int8_t *qs, const uint16_t *d, int64_t row_blocks, int64_t rows, int32_t k,
                          int32_t n_proj, const qk_proj_id16 *projs, const int32_t *counts, const int32_t *offsets,
                          const int32_t *items, void *ws, size_t ws_bytes, qk_stream stream) {
    return mmq_id_common(qs, d, row_blocks, rows, k, n_proj, projs, counts, offsets, items, ws, ws_bytes, true, stream);
}

// ------------------------------------------------------------------ the 4-bit key/value cache
static bool kv_shape(int32_t page_tokens, int32_t n_kv_heads, int32_t head_dim) {
    return page_tokens >= GROUP && page_tokens <= 4096 && page_tokens % GROUP == 0 && n_kv_heads >= 1 &&
           n_kv_heads <= 256 && (head_dim == 64 || head_dim == 128 || head_dim == 256);
}

size_t qk_kv_page_bytes(int32_t page_tokens, int32_t n_kv_heads, int32_t head_dim) {
    if (!kv_shape(page_tokens, n_kv_heads, head_dim)) return 0;
    return (size_t)page_tokens / GROUP * n_kv_heads * group_bytes(head_dim);
}

static qk_status check_cache(const qk_kv_cache *c) {
    REQUIRE(c, QK_ERR_ARG, "cache is null");
    REQUIRE(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256, QK_ERR_UNSUPPORTED,
            "head_dim=%d is not 64, 128 or 256", (int)c->head_dim);
    REQUIRE(kv_shape(c->page_tokens, c->n_kv_heads, c->head_dim), QK_ERR_ARG,
            "page_tokens=%d (a multiple of 16, 16..4096) or n_kv_heads=%d (1..256) out of range", (int)c->page_tokens,
            (int)c->n_kv_heads);
    REQUIRE(c->n_pages >= 1 && c->n_pages <= INT32_MAX / c->page_tokens, QK_ERR_ARG,
            "n_pages=%lld out of range (n_pages * page_tokens <= 2^31 - 1)", (long long)c->n_pages);
    REQUIRE(c->pages && aligned(c->pages, 16), QK_ERR_ARG, "pages is null or not 16-byte aligned");
    return QK_OK;
}
static Span cache_span(const qk_kv_cache *c) {
    return span(c->pages, (size_t)c->n_pages * qk_kv_page_bytes(c->page_tokens, c->n_kv_heads, c->head_dim));
}
static bool elem_ok(int32_t e) { return e == QK_ELEM_F32 || e == QK_ELEM_BF16; }
static unsigned elem_bytes(int32_t e) { return e == QK_ELEM_F32 ? 4 : 2; }
constexpr int64_t MOST_STRIDE = INT64_C(1) << 36;   // 2^24 rows * stride * 4 bytes stay inside 64 bits

qk_status qk_kv_append(const qk_kv_cache *cache, qk_elem elem, const void *q, int64_t q_stride, int32_t n_heads,
                       const void *k, int64_t k_stride, const void *v, int64_t v_stride, int64_t T, const int32_t *slots,
                       const qk_rope *rope, qk_elem q_elem, void *q_out, int64_t q_out_stride,
                       const int32_t *d_live_rows, qk_stream stream) {
    const qk_status st = check_cache(cache);
    if (st != QK_OK) return st;
    const int64_t D = cache->head_dim, kv = D * cache->n_kv_heads, qw = D * n_heads;
    REQUIRE(elem_ok(elem) && elem_ok(q_elem), QK_ERR_ARG, "bad element type");
    REQUIRE(T >= 0 && T <= (1 << 24), QK_ERR_ARG, "T=%lld out of range (0..2^24)", (long long)T);
    REQUIRE(n_heads >= 0 && n_heads <= 1024, QK_ERR_ARG, "n_heads=%d out of range", (int)n_heads);
    REQUIRE((k && v && slots) || T == 0, QK_ERR_ARG, "k, v or slots is null");
    REQUIRE(n_heads == 0 || T == 0 || (q && q_out), QK_ERR_ARG, "q or q_out is null");
    const unsigned e = elem_bytes(elem), qe = elem_bytes(q_elem);
    REQUIRE(aligned(k, e) && aligned(v, e) && aligned(slots, 4) && (n_heads == 0 || (aligned(q, e) && aligned(q_out, qe))),
            QK_ERR_ARG, "misaligned pointer");
    REQUIRE(k_stride >= kv && v_stride >= kv && (n_heads == 0 || (q_stride >= qw && q_out_stride >= qw)), QK_ERR_SHAPE,
            "a stride is smaller than its heads");
    REQUIRE(k_stride <= MOST_STRIDE && v_stride <= MOST_STRIDE &&
                (n_heads == 0 || (q_stride <= MOST_STRIDE && q_out_stride <= MOST_STRIDE)),
            QK_ERR_ARG, "a stride is out of range");
    KvRope r = {};
    if (rope) {
        REQUIRE(rope->kind == QK_ROPE_HALVES || rope->kind == QK_ROPE_ADJACENT, QK_ERR_ARG, "bad rope kind %d",
                (int)rope->kind);
        REQUIRE(rope->dims >= 8 && rope->dims <= D && rope->dims % 8 == 0, QK_ERR_SHAPE,
                "rope dims=%d is not a multiple of 8 in 8..head_dim", (int)rope->dims);
        REQUIRE(rope->n_axes >= 1 && rope->n_axes <= 4, QK_ERR_ARG, "n_axes=%d not in 1..4", (int)rope->n_axes);
        REQUIRE((rope->positions && rope->freqs) || T == 0, QK_ERR_ARG, "positions or freqs is null");
        REQUIRE(aligned(rope->positions, 4) && aligned(rope->freqs, 4), QK_ERR_ARG, "positions or freqs misaligned");
        r = {rope->kind, rope->dims, rope->n_axes, rope->positions, rope->freqs};
    }
    if (T == 0) return QK_OK;
    const Span outs[2] = {cache_span(cache), span(n_heads ? q_out : nullptr, n_heads ? rows_span(T, q_out_stride * qe, qw * qe) : 0)};
    const Span ins[7] = {span(n_heads ? q : nullptr, n_heads ? rows_span(T, q_stride * e, qw * e) : 0),
                         span(k, rows_span(T, k_stride * e, kv * e)),
                         span(v, rows_span(T, v_stride * e, kv * e)),
                         span(slots, (size_t)T * 4),
                         span(r.positions, (size_t)r.n_axes * T * 4),
                         span(r.freqs, (size_t)r.n_axes * (r.dims / 2) * 4),
                         span(d_live_rows, d_live_rows ? 4 : 0)};
    REQUIRE(!overlap(outs[0], outs[1]), QK_ERR_ALIAS, "q_out overlaps the cache");
    for (const Span &o : outs)
        for (const Span &i : ins) REQUIRE(!overlap(o, i), QK_ERR_ALIAS, "the cache or q_out overlaps an input");
    return launch_kv_append(kv_cache(cache), elem, q, q_stride, n_heads, k, k_stride, v, v_stride, (int)T, slots, r, q_elem,
                            q_out, q_out_stride, d_live_rows, (cudaStream_t)stream);
}

qk_status qk_kv_read(const qk_kv_cache *cache, const int32_t *slots, int64_t n, qk_elem elem, void *out,
                     int64_t out_stride, const int32_t *d_live_rows, qk_stream stream) {
    const qk_status st = check_cache(cache);
    if (st != QK_OK) return st;
    const int64_t width = 2LL * cache->n_kv_heads * cache->head_dim;
    REQUIRE(elem_ok(elem), QK_ERR_ARG, "bad element type %d", (int)elem);
    REQUIRE(n >= 0 && n <= (1 << 24), QK_ERR_ARG, "n=%lld out of range (0..2^24)", (long long)n);
    REQUIRE((slots && out) || n == 0, QK_ERR_ARG, "slots or out is null");
    REQUIRE(aligned(slots, 4) && aligned(out, elem_bytes(elem)), QK_ERR_ARG, "misaligned pointer");
    REQUIRE(out_stride >= width, QK_ERR_SHAPE, "out_stride=%lld < %lld", (long long)out_stride, (long long)width);
    REQUIRE(out_stride <= MOST_STRIDE, QK_ERR_ARG, "out_stride is out of range");
    if (n == 0) return QK_OK;
    const Span so = span(out, rows_span(n, out_stride * elem_bytes(elem), width * elem_bytes(elem)));
    REQUIRE(!overlap(so, cache_span(cache)) && !overlap(so, span(slots, (size_t)n * 4)) &&
                !overlap(so, span(d_live_rows, d_live_rows ? 4 : 0)),
            QK_ERR_ALIAS, "out overlaps an input");
    return launch_kv_read(kv_cache(cache), slots, (int)n, elem, out, out_stride, d_live_rows, (cudaStream_t)stream);
}

// ------------------------------------------------------------------ attention
constexpr int32_t MOST_KEYS = 1 << 30;   // of a sequence: places of keys stay inside an int
struct AttnSpans {
    Span in[6], out;
};
// What both calls have in common: rows of q and out, the page table of B sequences.
static qk_status check_attn(const qk_kv_cache *cache, const qk_attn *a, int64_t B, int64_t rows, bool image,
                            int64_t row_blocks, const int32_t *live, AttnSpans *sp) {
    REQUIRE(a, QK_ERR_ARG, "attn is null");
    REQUIRE(elem_ok(a->q_elem) && (!a->out || elem_ok(a->out_elem)), QK_ERR_ARG, "bad element type");
    REQUIRE(a->n_heads >= 1 && a->n_heads <= 1024 && a->n_heads % cache->n_kv_heads == 0, QK_ERR_UNSUPPORTED,
            "n_heads=%d is not a multiple of n_kv_heads=%d up to 1024", (int)a->n_heads, (int)cache->n_kv_heads);
    REQUIRE(std::isfinite(a->scale) && a->scale > 0.0f, QK_ERR_ARG, "scale must be positive and finite");
    REQUIRE(a->window >= 0, QK_ERR_ARG, "window < 0");
    const bool none = rows == 0 || B == 0;
    REQUIRE(none || (a->q && a->page_table && a->kv_lens), QK_ERR_ARG, "q, page_table or kv_lens is null");
    REQUIRE(none || a->out || image, QK_ERR_ARG, "neither out nor an image is wanted");
    const unsigned qe = elem_bytes(a->q_elem), oe = elem_bytes(a->out_elem);
    REQUIRE(aligned(a->q, qe) && aligned(a->out, oe) && aligned(a->page_table, 4) && aligned(a->kv_lens, 4) &&
                aligned(a->sinks, 4),
            QK_ERR_ARG, "misaligned pointer");
    const int64_t width = (int64_t)a->n_heads * cache->head_dim;
    REQUIRE(a->q_stride >= width && (!a->out || a->out_stride >= width), QK_ERR_SHAPE, "a stride is smaller than its heads");
    REQUIRE(a->q_stride <= MOST_STRIDE && (!a->out || a->out_stride <= MOST_STRIDE), QK_ERR_ARG, "a stride is out of range");
    REQUIRE(a->table_stride >= 1 && a->table_stride <= MOST_KEYS / cache->page_tokens, QK_ERR_ARG,
            "table_stride=%lld out of range (table_stride * page_tokens <= 2^30)", (long long)a->table_stride);
    REQUIRE(!image || row_blocks >= width / QB, QK_ERR_SHAPE, "the image row (%lld blocks) is smaller than the heads",
            (long long)row_blocks);
    REQUIRE(!image || row_blocks <= (1 << 20), QK_ERR_ARG, "image row blocks > 2^20");
    sp->in[0] = cache_span(cache);
    sp->in[1] = span(a->q, rows_span(rows, a->q_stride * qe, width * qe));
    sp->in[2] = span(a->page_table, (size_t)(B * a->table_stride * 4));
    sp->in[3] = span(a->kv_lens, (size_t)B * 4);
    sp->in[4] = span(a->sinks, a->sinks ? (size_t)a->n_heads * 4 : 0);
    sp->in[5] = span(live, live ? 4 : 0);
    sp->out = span(a->out, a->out ? rows_span(rows, a->out_stride * oe, width * oe) : 0);
    REQUIRE(none || std::none_of(sp->in, sp->in + 6, [&](Span i) { return overlap(sp->out, i); }), QK_ERR_ALIAS,
            "out overlaps an input");
    return QK_OK;
}

size_t qk_attn_decode_workspace_bytes(const qk_kv_cache *cache, int32_t n_heads, int64_t B, int32_t T) {
    if (!cache || !kv_shape(cache->page_tokens, cache->n_kv_heads, cache->head_dim) || n_heads < 1 || n_heads > 1024 ||
        n_heads % cache->n_kv_heads || B < 0 || B > (1 << 20) || T < 1 || T > 8)
        return 0;
    return (size_t)attn_decode_workspace_bytes(cache->n_kv_heads, cache->head_dim, n_heads, B, T);
}

qk_status qk_attn_decode(const qk_kv_cache *cache, const qk_attn *attn, int64_t B, int32_t T, void *img,
                         int64_t img_row_blocks, const int32_t *d_live_rows, void *ws, size_t ws_bytes, qk_stream stream) {
    qk_status st = check_cache(cache);
    if (st != QK_OK) return st;
    REQUIRE(B >= 0 && B <= (1 << 20), QK_ERR_ARG, "B=%lld out of range (0..2^20)", (long long)B);
    REQUIRE(T >= 1, QK_ERR_ARG, "T < 1");
    REQUIRE(T <= 8, QK_ERR_UNSUPPORTED, "T=%d > 8 (use qk_attn_prefill)", (int)T);
    REQUIRE(!attn || B * T * (int64_t)attn->n_heads <= INT32_MAX, QK_ERR_UNSUPPORTED, "B * T * n_heads too large for one launch");
    AttnSpans sp;
    st = check_attn(cache, attn, B, B * T, img != nullptr, img_row_blocks, d_live_rows, &sp);
    if (st != QK_OK) return st;
    REQUIRE(aligned(img, 4), QK_ERR_ARG, "img not 4-byte aligned");
    if (B == 0) return QK_OK;
    const Span si = span(img, img ? (size_t)(B * T * img_row_blocks * Q8_1_BYTES) : 0);
    const size_t need = qk_attn_decode_workspace_bytes(cache, attn->n_heads, B, T);
    REQUIRE(ws && aligned(ws, 16), QK_ERR_WORKSPACE, "workspace null or not 16-byte aligned");
    REQUIRE(ws_bytes >= need, QK_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    const Span sw = span(ws, need);
    REQUIRE(!overlap(si, sp.out) && !overlap(sw, si) && !overlap(sw, sp.out), QK_ERR_ALIAS,
            "out, img and the workspace overlap");
    for (const Span &i : sp.in)
        REQUIRE(!overlap(si, i) && !overlap(sw, i), QK_ERR_ALIAS, "img or the workspace overlaps an input");
    qk_attn a = *attn;
    if (a.window >= MOST_KEYS) a.window = 0;   // no sequence has as many
    return launch_attn_decode(kv_cache(cache), a, (int)B, T, static_cast<uint8_t *>(img), img_row_blocks, d_live_rows,
                              ws, (cudaStream_t)stream);
}

size_t qk_attn_prefill_workspace_bytes(const qk_kv_cache *cache, int64_t B, int64_t max_kv) {
    if (!cache || !kv_shape(cache->page_tokens, cache->n_kv_heads, cache->head_dim) || B < 0 || B > 65535 || max_kv < 1 ||
        max_kv > INT32_MAX)
        return 0;
    return (size_t)attn_prefill_workspace_bytes(cache->n_kv_heads, cache->head_dim, B, max_kv);
}

qk_status qk_attn_prefill(const qk_kv_cache *cache, const qk_attn *attn, int64_t B, int64_t rows,
                          const int32_t *q_offsets, int64_t max_kv, int8_t *qs, uint16_t *d, int64_t row_blocks,
                          const int32_t *d_live_rows, void *ws, size_t ws_bytes, qk_stream stream) {
    qk_status st = check_cache(cache);
    if (st != QK_OK) return st;
    REQUIRE(B >= 0 && rows >= 0, QK_ERR_ARG, "B or rows < 0");
    REQUIRE(B <= 65535 && rows <= (1 << 24), QK_ERR_UNSUPPORTED, "B=%lld > 65535 or rows=%lld > 2^24", (long long)B,
            (long long)rows);
    REQUIRE((qs != nullptr) == (d != nullptr), QK_ERR_ARG, "one of qs and d is null");
    AttnSpans sp;
    st = check_attn(cache, attn, B, rows, qs != nullptr, row_blocks, d_live_rows, &sp);
    if (st != QK_OK) return st;
    REQUIRE(max_kv >= 1 && max_kv <= attn->table_stride * cache->page_tokens, QK_ERR_ARG,
            "max_kv=%lld not in 1..table_stride * page_tokens", (long long)max_kv);
    REQUIRE(aligned(qs, 16) && aligned(d, 4) && aligned(q_offsets, 4), QK_ERR_ARG,
            "misaligned pointer (qs must be 16-byte, d 4-byte aligned)");
    if (B == 0 || rows == 0) return QK_OK;
    REQUIRE(q_offsets, QK_ERR_ARG, "q_offsets is null");
    // rows of the staged keys and values are counted in int, and so are the CTAs
    REQUIRE(B * cache->n_kv_heads * (max_kv + 127) < (1LL << 31) && B * cache->n_kv_heads * cache->head_dim < (1LL << 31) &&
                (rows + 256 * B) * attn->n_heads < (1LL << 31),
            QK_ERR_UNSUPPORTED, "B * n_kv_heads * max_kv or rows * n_heads too large for one launch");
    const size_t need = qk_attn_prefill_workspace_bytes(cache, B, max_kv);
    REQUIRE(ws && aligned(ws, 128), QK_ERR_WORKSPACE, "workspace null or not 128-byte aligned");
    REQUIRE(ws_bytes >= need, QK_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws_bytes, need);
    const Span outs[4] = {sp.out, span(qs, qs ? (size_t)(rows * row_blocks * QB) : 0),
                          span(d, d ? (size_t)(rows * row_blocks * 2) : 0), span(ws, need)};
    for (int o = 0; o < 4; o++) {
        for (const Span &i : sp.in) REQUIRE(!overlap(outs[o], i), QK_ERR_ALIAS, "an output or the workspace overlaps an input");
        REQUIRE(!overlap(outs[o], span(q_offsets, (size_t)(B + 1) * 4)), QK_ERR_ALIAS,
                "an output or the workspace overlaps q_offsets");
        for (int i = 0; i < o; i++) REQUIRE(!overlap(outs[o], outs[i]), QK_ERR_ALIAS, "outputs and the workspace overlap");
    }
    qk_attn a = *attn;
    if (a.window >= MOST_KEYS) a.window = 0;   // no sequence has as many
    return launch_attn_prefill(kv_cache(cache), a, (int)B, (int)rows, q_offsets, (int)max_kv, qs, d, row_blocks,
                               d_live_rows, ws, (cudaStream_t)stream);
}

}  // extern "C"

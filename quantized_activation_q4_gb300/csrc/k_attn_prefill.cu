// Attention over the 4-bit key/value cache, its output's Q8 image beside the rows.
//
// One warp per (query row, head): lane l holds columns 32 b + l of the query and of the output, keys one after another
// with a running maximum and sum.

#include "qk_kv.cuh"

namespace qk {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E = 1.4426950408889634f;

struct Rows {   // decode: T rows a sequence; prefill: offsets
    int B, T, rows, max_kv;
    const int32_t *offsets;
};
struct Image {
    uint8_t *img;    // Q8_1 blocks
    int8_t *qs;      // or Q8_0 planes
    uint16_t *d;
    int64_t row_blocks;
};

__device__ __forceinline__ float load_q(const void *q, int elem, int64_t at) {
    if (elem == QK_ELEM_F32) return ld_prev(static_cast<const float *>(q) + at);
    return __uint_as_float((uint32_t)ld_prev(static_cast<const uint16_t *>(q) + at) << 16);
}

template <int NB>
__global__ void __launch_bounds__(128) attn_rows_kernel(KvCache c, qk_attn a, Rows R, Image im, const int32_t *live) {
    pdl_trigger();
    pdl_wait();
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, D = 32 * NB;
    const int row = (int)(unit / a.n_heads), head = (int)(unit % a.n_heads);
    if (row >= R.rows) return;
    int b, i, n;
    if (R.offsets) {
        b = -1;
        for (int s = 0; s < R.B; s++) {
            const int lo = min(max(ld_prev(R.offsets + s), 0), R.rows), hi = min(max(ld_prev(R.offsets + s + 1), 0), R.rows);
            if (row >= lo && row < hi) {
                b = s;
                i = row - lo;
                n = hi - lo;
                break;
            }
        }
        if (b < 0) return;
    } else {
        b = row / R.T;
        i = row % R.T;
        n = R.T;
    }
    if (b >= live_rows(live, R.B)) return;
    const int64_t most = min((int64_t)R.max_kv, a.table_stride * c.page_tokens);
    const int len = (int)min((int64_t)max(ld_prev(a.kv_lens + b), 0), most);
    const int end = len - n + i + 1;
    const int begin = a.window > 0 ? max(0, end - a.window) : 0;
    const int kv_head = head / (a.n_heads / c.Hkv);
    float q[NB], o[NB];
#pragma unroll
    for (int k = 0; k < NB; k++) {
        q[k] = load_q(a.q, a.q_elem, row * a.q_stride + (int64_t)head * D + 32 * k + lane) * (a.scale * LOG2E);
        o[k] = 0.0f;
    }
    float top = -INFINITY, sum = 0.0f;
    for (int j = begin; j < end; j++) {
        const int page = ld_prev(a.page_table + b * a.table_stride + j / c.page_tokens);
        if (page < 0 || page >= c.n_pages) continue;
        const int in_page = j % c.page_tokens, i16 = in_page % GROUP;
        const uint8_t *g = group_at(c, page, kv_head, in_page);
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NB; k++) {
            const int w = ld_prev(g + k_word_at(D, i16, k, lane % 16 / 4) + lane % 4);
            const float d = __half2float(__ushort_as_half(ld_prev(reinterpret_cast<const uint16_t *>(g + k_scale_at(D, i16, k)))));
            s = fmaf((float)((lane < 16 ? w & 15 : w >> 4) - 8) * d, q[k], s);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(FULL, s, m);
        const float now = fmaxf(top, s), old = exp2f(top - now), p = exp2f(s - now);
        top = now;
        sum = sum * old + p;
#pragma unroll
        for (int k = 0; k < NB; k++) {
            const int w = ld_prev(g + v_byte_at(D, i16, 2 * k + lane / 16, lane % 8));
            const float d = __half2float(__ushort_as_half(ld_prev(reinterpret_cast<const uint16_t *>(g + v_scale_at(D, i16, k)))));
            o[k] = fmaf((float)((lane % 16 < 8 ? w & 15 : w >> 4) - 8) * d, p, o[k] * old);
        }
    }
    if (a.sinks) {
        const float s = ld_prev(a.sinks + head) * LOG2E, now = fmaxf(top, s);
        const float old = top == -INFINITY ? 0.0f : exp2f(top - now);
        sum = sum * old + exp2f(s - now);
#pragma unroll
        for (int k = 0; k < NB; k++) o[k] *= old;
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int k = 0; k < NB; k++) {
        const float y = o[k] * inv;
        const int64_t at = row * a.out_stride + (int64_t)head * D + 32 * k + lane;
        if (a.out && a.out_elem == QK_ELEM_F32) static_cast<float *>(a.out)[at] = y;
        if (a.out && a.out_elem == QK_ELEM_BF16) static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
        float m = fabsf(y);
#pragma unroll
        for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, x));
        const float d = m / 127.0f;
        const int code = m != 0.0f ? __float2int_rn(y / d) : 0;
        int total = code;
#pragma unroll
        for (int x = 16; x; x >>= 1) total += __shfl_xor_sync(FULL, total, x);
        const int64_t block = row * im.row_blocks + head * NB + k;
        if (im.img) {
            im.img[block * Q8_1_BYTES + 4 + lane] = (uint8_t)code;
            if (lane == 0)
                *reinterpret_cast<__half2 *>(im.img + block * Q8_1_BYTES) =
                    __halves2half2(__float2half_rn(d), __float2half_rn(d * (float)total));
        }
        if (im.qs) {
            im.qs[block * QB + lane] = (int8_t)code;
            if (lane == 0) im.d[block] = __half_as_ushort(__float2half_rn(d));
        }
    }
    if (head == a.n_heads - 1)   // the blocks behind the heads
        for (int64_t block = row * im.row_blocks + a.n_heads * NB; block < (row + 1) * im.row_blocks; block++) {
            if (im.img) {
                im.img[block * Q8_1_BYTES + 4 + lane] = 0;
                if (lane == 0) *reinterpret_cast<uint32_t *>(im.img + block * Q8_1_BYTES) = 0;
            }
            if (im.qs) {
                im.qs[block * QB + lane] = 0;
                if (lane == 0) im.d[block] = 0;
            }
        }
}

qk_status launch_rows(const KvCache &c, const qk_attn &a, const Rows &R, const Image &im, const int32_t *live,
                      cudaStream_t s) {
    const dim3 grid((unsigned)ceil_div((int64_t)R.rows * a.n_heads, 4));
    auto *kernel = c.D == 64 ? attn_rows_kernel<2> : c.D == 128 ? attn_rows_kernel<4> : attn_rows_kernel<8>;
    return launch_pdl("attn", kernel, grid, dim3(128), 0, s, c, a, R, im, live);
}

}  // namespace

int64_t attn_prefill_workspace_bytes(int, int, int64_t, int64_t) { return 128; }

qk_status launch_attn_prefill(const KvCache &c, const qk_attn &a, int B, int rows, const int32_t *q_offsets, int max_kv,
                              int8_t *qs, uint16_t *d, int64_t row_blocks, const int32_t *live, void *, cudaStream_t s) {
    return launch_rows(c, a, {B, 0, rows, max_kv, q_offsets}, {nullptr, qs, d, row_blocks}, live, s);
}

}  // namespace qk

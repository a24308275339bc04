// Writing to and reading from the 4-bit key/value cache.
//
//   kv_append_kernel  q, k and v rows of one token: rotation by positions, q to rows, k and v to 4-bit blocks
//   kv_read_kernel    the values of cached tokens as rows
//
// Both are bound by memory: append reads a token's q, k and v rows once, writes q once and 9/16 byte a cached value.
// A block of 32 columns is handled by 8 consecutive lanes, 4 columns each; its codes meet their nibble partners by one
// shuffle (columns 16 apart for k, 8 apart for v). Arithmetic is binary32 with IEEE division.

#include "qk_kv.cuh"

namespace qk {
namespace {

constexpr unsigned FULL = 0xffffffffu;

// ---------------------------------------------------------------- angles
// The fraction of a turn that positions * freqs come to, as a sum hi + lo with |hi| <= 1/2 and lo below its last place.
// A frequency in turns (times 1 / (2 pi)) is held in three floats, and a position in two parts that binary32 holds
// exactly; their products are split exactly into a rounded value and its rest, and the whole turns of every part drop
// out without error. So the fraction of any int32 position is right to about 2^-26 turns, where a binary32 angle would
// be wrong by 2^-24 of itself: 0.06 rad at position 10^6.
struct Turn {
    float hi, lo;
};
__device__ __forceinline__ void add_fraction(Turn &s, float w) {
    const float f = w - rintf(w);
    const float sum = s.hi + f, back = sum - s.hi;   // two-sum
    s.lo += (s.hi - (sum - back)) + (f - back);
    s.hi = sum;
}
__device__ __forceinline__ void add_product(Turn &s, float m, const float t[3]) {
    const float w = m * t[0], w2 = m * t[1];
    add_fraction(s, w);
    add_fraction(s, fmaf(m, t[0], -w));
    add_fraction(s, w2);
    s.lo += fmaf(m, t[2], fmaf(m, t[1], -w2));
}
__device__ __forceinline__ Turn turn_of(const KvRope &r, int T, int t, int pair) {
    constexpr float C0 = 0.159154937f, C1 = 6.42063824e-09f, C2 = 7.3427387e-17f;   // 1 / (2 pi)
    Turn s = {0.0f, 0.0f};
    for (int a = 0; a < r.n_axes; a++) {
        const int p = ld_prev(r.positions + (int64_t)a * T + t);
        const float f = ld_prev(r.freqs + a * (r.dims / 2) + pair);
        // f / (2 pi) in three floats
        const float p0 = f * C0, e0 = fmaf(f, C0, -p0), p1 = f * C1, e1 = fmaf(f, C1, -p1);
        const float sum = e0 + p1, back = sum - e0;
        const float turns[3] = {p0, sum, (e0 - (sum - back)) + (p1 - back) + fmaf(f, C2, e1)};
        add_product(s, (float)(p >> 12) * 4096.0f, turns);
        add_product(s, (float)(p & 4095), turns);
    }
    s.hi -= rintf(s.hi);
    const float h = s.hi + s.lo, l = s.lo - (h - s.hi);
    return {h - rintf(h), l};
}
__device__ __forceinline__ float2 cos_sin(Turn u) {
    float sn, cs;
    sincospif(2.0f * u.hi, &sn, &cs);
    const float e = u.lo * 6.2831855f;
    return make_float2(fmaf(-sn, e, cs), fmaf(cs, e, sn));
}

// ---------------------------------------------------------------- 4-bit blocks
// One block held by 8 lanes (4 values each, j8 the lane's index); all lanes of the warp call. Codes in the bytes of
// the result, the scale in *d.
__device__ __forceinline__ uint32_t q4_block(float4 x, int j8, float *d) {
    const float v[4] = {x.x, x.y, x.z, x.w};
    float a = fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))), 0.0f);
    a = fmaxf(a, __shfl_xor_sync(FULL, a, 1));
    a = fmaxf(a, __shfl_xor_sync(FULL, a, 2));
    a = fmaxf(a, __shfl_xor_sync(FULL, a, 4));
    int first = 64;   // 2 * column + sign of the first value of that magnitude
#pragma unroll
    for (int i = 3; i >= 0; i--)
        if (fabsf(v[i]) == a) first = 2 * (4 * j8 + i) + (v[i] < 0.0f);
    first = min(first, __shfl_xor_sync(FULL, first, 1));
    first = min(first, __shfl_xor_sync(FULL, first, 2));
    first = min(first, __shfl_xor_sync(FULL, first, 4));
    const float size = fminf(a * 0.125f, 65504.0f);
    *d = (first & 1) ? size : -size;
    uint32_t codes = 0x08080808u;
    if (size != 0.0f) {
        codes = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int c = min(max(__float2int_rn(v[i] / *d), -8), 7) + 8;
            codes |= (uint32_t)c << (8 * i);
        }
    }
    return codes;
}
__device__ __forceinline__ uint16_t half_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }

// ---------------------------------------------------------------- append
// CTA (t, y) takes every gridDim.y-th share of token t's heads: q heads, then k, then v, four columns to a lane.
template <typename X, typename Q>
__global__ void __launch_bounds__(256) kv_append_kernel(KvCache c, const X *q, int64_t q_stride, int n_heads, const X *k,
                                                        int64_t k_stride, const X *v, int64_t v_stride, int T,
                                                        const int32_t *slots, KvRope rope, Q *q_out,
                                                        int64_t q_out_stride, bool wide, bool q_wide,
                                                        const int32_t *live) {
    __shared__ float2 cs[128];
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x, D = c.D;
    if (t >= live_rows(live, T)) return;
    const int half = rope.dims / 2;
    for (int i = threadIdx.x; i < half; i += blockDim.x) cs[i] = cos_sin(turn_of(rope, T, t, i));
    __syncthreads();
    const int slot = ld_prev(slots + t);
    const bool stored = slot >= 0 && slot / c.page_tokens < c.n_pages;
    const int page = stored ? slot / c.page_tokens : 0, in_page = stored ? slot % c.page_tokens : 0, i16 = in_page % GROUP;
    const int quads = D / 4, total = (n_heads + 2 * c.Hkv) * quads;
    for (int base = (blockIdx.y * 8 + (threadIdx.x >> 5)) * 32; base < total; base += gridDim.y * 256) {
        const int u = base + (threadIdx.x & 31);
        const int head = u < total ? u / quads : 0, x0 = u < total ? (u % quads) * 4 : 0;
        const bool is_q = head < n_heads, is_k = !is_q && head < n_heads + c.Hkv;
        const int kv_head = is_q ? 0 : is_k ? head - n_heads : head - n_heads - c.Hkv;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (u < total) {
            const X *row = is_q   ? q + t * q_stride + (int64_t)head * D
                           : is_k ? k + t * k_stride + (int64_t)kv_head * D
                                  : v + t * v_stride + (int64_t)kv_head * D;
            x = load_row4(row + x0, wide);
            if ((is_q || is_k) && x0 < rope.dims) {
                if (rope.kind == QK_ROPE_ADJACENT) {
                    const float2 a = cs[x0 / 2], b = cs[x0 / 2 + 1];
                    x = make_float4(x.x * a.x - x.y * a.y, x.y * a.x + x.x * a.y, x.z * b.x - x.w * b.y,
                                    x.w * b.x + x.z * b.y);
                } else {   // the partners are half the rotated columns away
                    const bool low = x0 < half;
                    const float4 y = load_row4(row + (low ? x0 + half : x0 - half), wide);
                    const float2 *a = cs + (low ? x0 : x0 - half);
                    const float sg = low ? -1.0f : 1.0f;
                    x = make_float4(x.x * a[0].x + sg * (y.x * a[0].y), x.y * a[1].x + sg * (y.y * a[1].y),
                                    x.z * a[2].x + sg * (y.z * a[2].y), x.w * a[3].x + sg * (y.w * a[3].y));
                }
            }
            if (is_q) store_row4(q_out + t * q_out_stride + (int64_t)head * D + x0, x, q_wide);
        }
        if (base + 31 < n_heads * quads) continue;   // the whole warp holds q
        const int j8 = threadIdx.x & 7, b = x0 / 32;
        float d;
        const uint32_t codes = q4_block(x, j8, &d);
        const uint32_t k_hi = __shfl_down_sync(FULL, codes, 4), v_hi = __shfl_down_sync(FULL, codes, 2);
        if (u >= total || is_q || !stored) continue;
        uint8_t *g = group_at(c, page, kv_head, in_page);
        if (is_k) {
            if (j8 < 4) *reinterpret_cast<uint32_t *>(g + k_word_at(D, i16, b, j8)) = codes | k_hi << 4;
            if (j8 == 0) *reinterpret_cast<uint16_t *>(g + k_scale_at(D, i16, b)) = half_bits(d);
        } else {
            if ((j8 & 2) == 0) {
                const uint32_t w = codes | v_hi << 4;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    g[v_byte_at(D, i16, 2 * b + (j8 >> 2), 4 * (j8 & 1) + e)] = (uint8_t)(w >> (8 * e));
            }
            if (j8 == 0) *reinterpret_cast<uint16_t *>(g + v_scale_at(D, i16, b)) = half_bits(d);
        }
    }
}

// ---------------------------------------------------------------- read
// Four columns to a thread.
template <typename Y>
__global__ void __launch_bounds__(256) kv_read_kernel(KvCache c, const int32_t *slots, int n, Y *out, int64_t out_stride,
                                                      bool wide, const int32_t *live) {
    pdl_trigger();
    pdl_wait();
    const int r = blockIdx.x, D = c.D;
    if (r >= live_rows(live, n)) return;
    const int slot = ld_prev(slots + r);
    if (slot < 0 || slot / c.page_tokens >= c.n_pages) return;
    const int page = slot / c.page_tokens, in_page = slot % c.page_tokens, i16 = in_page % GROUP;
    const int quads = D / 4, total = 2 * c.Hkv * quads;
    for (int u = blockIdx.y * 256 + threadIdx.x; u < total; u += gridDim.y * 256) {
        const int head = u / quads, x0 = (u % quads) * 4, b = x0 / 32;
        const bool is_k = head < c.Hkv;
        const uint8_t *g = group_at(c, page, is_k ? head : head - c.Hkv, in_page);
        uint32_t w;
        if (is_k) {
            w = ld_prev(reinterpret_cast<const uint32_t *>(g + k_word_at(D, i16, b, x0 % 16 / 4)));
            w >>= x0 % 32 < 16 ? 0 : 4;
        } else {
            w = 0;
#pragma unroll
            for (int e = 0; e < 4; e++)
                w |= (uint32_t)ld_prev(g + v_byte_at(D, i16, x0 / 16, x0 % 8 + e)) << (8 * e);
            w >>= x0 % 16 < 8 ? 0 : 4;
        }
        const uint16_t d =
            ld_prev(reinterpret_cast<const uint16_t *>(g + (is_k ? k_scale_at(D, i16, b) : v_scale_at(D, i16, b))));
        const float df = __half2float(__ushort_as_half(d));
        const float4 x = make_float4((float)((int)(w & 15) - 8) * df, (float)((int)(w >> 8 & 15) - 8) * df,
                                     (float)((int)(w >> 16 & 15) - 8) * df, (float)((int)(w >> 24 & 15) - 8) * df);
        store_row4(out + r * out_stride + (int64_t)head * D + x0, x, wide);
    }
}

}  // namespace

qk_status launch_kv_append(const KvCache &c, int elem, const void *q, int64_t q_stride, int n_heads, const void *k,
                           int64_t k_stride, const void *v, int64_t v_stride, int T, const int32_t *slots,
                           const KvRope &rope, int q_elem, void *q_out, int64_t q_out_stride, const int32_t *live,
                           cudaStream_t s) {
    const int total = (n_heads + 2 * c.Hkv) * (c.D / 4);
    const dim3 grid(T, (unsigned)ceil_div(total, 256 * 4));
    const bool wide = row_wide(k, k_stride, elem) && row_wide(v, v_stride, elem) && (n_heads == 0 || row_wide(q, q_stride, elem));
    const bool q_wide = row_wide(q_out, q_out_stride, q_elem);
    const auto go = [&](auto x, auto y) {
        using X = decltype(x);
        using Q = decltype(y);
        return launch_pdl("kv_append", kv_append_kernel<X, Q>, grid, dim3(256), 0, s, c, static_cast<const X *>(q),
                          q_stride, n_heads, static_cast<const X *>(k), k_stride, static_cast<const X *>(v), v_stride, T,
                          slots, rope, static_cast<Q *>(q_out), q_out_stride, wide, q_wide, live);
    };
    if (elem == QK_ELEM_F32) return q_elem == QK_ELEM_F32 ? go(float{}, float{}) : go(float{}, __nv_bfloat16{});
    return q_elem == QK_ELEM_F32 ? go(__nv_bfloat16{}, float{}) : go(__nv_bfloat16{}, __nv_bfloat16{});
}

qk_status launch_kv_read(const KvCache &c, const int32_t *slots, int n, int elem, void *out, int64_t out_stride,
                         const int32_t *live, cudaStream_t s) {
    const dim3 grid(n, (unsigned)ceil_div(2 * c.Hkv * (c.D / 4), 256));
    const bool wide = row_wide(out, out_stride, elem);
    if (elem == QK_ELEM_F32)
        return launch_pdl("kv_read", kv_read_kernel<float>, grid, dim3(256), 0, s, c, slots, n,
                          static_cast<float *>(out), out_stride, wide, live);
    return launch_pdl("kv_read", kv_read_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, c, slots, n,
                      static_cast<__nv_bfloat16 *>(out), out_stride, wide, live);
}

}  // namespace qk

// Writing to and reading from the 4-bit key/value cache.
//
//   kv_append_kernel  q, k and v rows of one token: rotation by positions, q to rows, k and v to 4-bit blocks
//   kv_read_kernel    the values of cached tokens as rows
//
// Append reads a token's q, k and v rows once, writes q once and 9/16 byte a cached value. 3325 tokens of 28 + 8 heads of 128
// with three axes: 25 us, 3.1 TB/s; 5000 warp instructions a token, issued 58% of the time; the largest stall is the barrier
// behind the angles, which few threads work out. Four quads a thread in any head 43 us, four tokens a CTA 65 (registers). Read of 16384 tokens of 8 heads: 21 us,
// 4.1 TB/s; one token and quad a thread 67.
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
    int at[4];
    float freq[4];
#pragma unroll
    for (int a = 0; a < 4; a++) {   // (all loads before the first use)
        at[a] = a < r.n_axes ? ld_prev(r.positions + (int64_t)a * T + t) : 0;
        freq[a] = a < r.n_axes ? ld_prev(r.freqs + a * (r.dims / 2) + pair) : 0.0f;
    }
#pragma unroll
    for (int a = 0; a < 4; a++) {
        const int p = at[a];
        const float f = freq[a];
        if (f == 0.0f) continue;   // the pair belongs to another axis
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
        const float inv = 1.0f / *d;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            // rint(v / d): the product with 1 / d is within 8 * 2^-22 of the quotient, so a division next to ties alone
            float q = v[i] * inv, c = rintf(q);
            if (!(fabsf(fabsf(q - c) - 0.5f) >= 1e-5f) || size < 0x1p-100f) c = rintf(v[i] / *d);
            c = c == c ? fminf(fmaxf(c, -8.0f), 7.0f) : 0.0f;
            codes |= (uint32_t)((int)c + 8) << (8 * i);
        }
    }
    return codes;
}
__device__ __forceinline__ uint16_t half_bits(float v) { return __half_as_ushort(__float2half_rn(v)); }

// ---------------------------------------------------------------- append
// One CTA a token: thread i has the quad of columns i % (D / 4) of every 256 / (D / 4)-th head, so its cosines, sines and
// places inside a head are the same for all of them. The first loads are under way before the angles are worked out.
constexpr int BATCH = 4;   // heads of q whose loads are under way together
template <int D, bool HALVES, typename X, typename Q>
__global__ void __launch_bounds__(256) kv_append_kernel(KvCache c, const X *q, int64_t q_stride, int n_heads, const X *k,
                                                        int64_t k_stride, const X *v, int64_t v_stride, int T,
                                                        const int32_t *slots, KvRope rope, Q *q_out,
                                                        int64_t q_out_stride, bool wide, bool q_wide,
                                                        const int32_t *live) {
    constexpr int QUADS = D / 4, HEADS = 256 / QUADS;
    __shared__ __align__(16) float2 cs[D / 2];
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x, half = rope.dims / 2;
    if (t >= live_rows(live, T)) return;
    const int slot = ld_prev(slots + t);
    const int x0 = threadIdx.x % QUADS * 4, h0 = threadIdx.x / QUADS;
    const bool turned = x0 < rope.dims, low = x0 < half;
    const int partner = HALVES && turned ? (low ? half : -half) : 0;
    const X *q_at = q + t * q_stride + x0;
    Q *q_to = q_out + t * q_out_stride + x0;

    float4 x[BATCH], y[BATCH];   // columns, and their partners in a rotation by halves
    const auto load_q = [&](int h) {
#pragma unroll
        for (int e = 0; e < BATCH; e++)
            if (h + e * HEADS < n_heads) {
                const X *row = q_at + (int64_t)(h + e * HEADS) * D;
                x[e] = load_row4(row, wide);
                if (HALVES) y[e] = load_row4(row + partner, wide);
            }
    };
    load_q(h0);
    for (int i = threadIdx.x; i < half; i += 256) cs[i] = cos_sin(turn_of(rope, T, t, i));
    __syncthreads();
    float cosine[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sine[4] = {};
    if (turned) {
        const float4 *f = reinterpret_cast<const float4 *>(cs + (HALVES ? (low ? x0 : x0 - half) : x0 / 2));
        const float4 f0 = f[0];
        if (HALVES) {
            const float4 f1 = f[1];
            cosine[0] = f0.x, cosine[1] = f0.z, cosine[2] = f1.x, cosine[3] = f1.z;
            sine[0] = f0.y, sine[1] = f0.w, sine[2] = f1.y, sine[3] = f1.w;
            if (low)
#pragma unroll
                for (int i = 0; i < 4; i++) sine[i] = -sine[i];
        } else {
            cosine[0] = f0.x, sine[0] = f0.y, cosine[1] = f0.z, sine[1] = f0.w;
        }
    }
    const auto rotated = [&](float4 a, float4 b) {
        if (!turned) return a;
        if (HALVES)
            return make_float4(fmaf(a.x, cosine[0], b.x * sine[0]), fmaf(a.y, cosine[1], b.y * sine[1]),
                               fmaf(a.z, cosine[2], b.z * sine[2]), fmaf(a.w, cosine[3], b.w * sine[3]));
        return make_float4(fmaf(a.x, cosine[0], -(a.y * sine[0])), fmaf(a.y, cosine[0], a.x * sine[0]),
                           fmaf(a.z, cosine[1], -(a.w * sine[1])), fmaf(a.w, cosine[1], a.z * sine[1]));
    };
    for (int h = h0; h < n_heads;) {
#pragma unroll
        for (int e = 0; e < BATCH; e++)
            if (h + e * HEADS < n_heads) store_row4(q_to + (int64_t)(h + e * HEADS) * D, rotated(x[e], y[e]), q_wide);
        h += BATCH * HEADS;
        load_q(h);
    }

    const bool stored = slot >= 0 && slot / c.page_tokens < c.n_pages;
    if (!stored) return;
    const int page = slot / c.page_tokens, in_page = slot - page * c.page_tokens, i16 = in_page % GROUP;
    const int j8 = threadIdx.x & 7, blk = x0 / 32;
    // whole warps take part in the blocks' shuffles
    for (int h = h0; h - (int)(threadIdx.x & 31) / QUADS < 2 * c.Hkv; h += HEADS) {
        const bool there = h < 2 * c.Hkv, is_k = h < c.Hkv;
        const int head = is_k ? h : h - c.Hkv;
        float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (there) {
            const X *row = (is_k ? k + t * k_stride : v + t * v_stride) + (int64_t)head * D + x0;
            r = load_row4(row, wide);
            if (is_k) r = rotated(r, HALVES ? load_row4(row + partner, wide) : r);
        }
        float d;
        const uint32_t codes = q4_block(r, j8, &d);
        const uint32_t k_hi = __shfl_down_sync(FULL, codes, 4), v_hi = __shfl_down_sync(FULL, codes, 2);
        if (!there) continue;
        uint8_t *g = group_at(c, page, head, in_page);
        if (is_k) {
            if (j8 < 4) *reinterpret_cast<uint32_t *>(g + k_word_at(D, i16, blk, j8)) = codes | k_hi << 4;
            if (j8 == 0) *reinterpret_cast<uint16_t *>(g + k_scale_at(D, i16, blk)) = half_bits(d);
        } else {
            if ((j8 & 2) == 0) {
                const uint32_t w = codes | v_hi << 4;
                uint8_t *to = g + v_byte_at(D, i16, 2 * blk + (j8 >> 2), 4 * (j8 & 1));
#pragma unroll
                for (int f = 0; f < 4; f++) to[64 * f] = (uint8_t)(w >> (8 * f));
            }
            if (j8 == 0) *reinterpret_cast<uint16_t *>(g + v_scale_at(D, i16, blk)) = half_bits(d);
        }
    }
}

// ---------------------------------------------------------------- read
// A thread takes a word of a k head (columns 4t .. and 16 + 4t .. of a block) or the bytes of eight columns of a v head
// (u .. u + 3 and u + 8 .. of a column tile), of READ_ROWS tokens, whose loads are under way together.
constexpr int READ_ROWS = 4;
__device__ __forceinline__ float4 code_values(uint32_t w, float d) {
    return make_float4((float)((int)(w & 15) - 8) * d, (float)((int)(w >> 8 & 15) - 8) * d, (float)((int)(w >> 16 & 15) - 8) * d,
                       (float)((int)(w >> 24 & 15) - 8) * d);
}
template <int D, typename Y>
__global__ void __launch_bounds__(256) kv_read_kernel(KvCache c, const int32_t *slots, int n, Y *out, int64_t out_stride,
                                                      bool wide, const int32_t *live) {
    pdl_trigger();
    pdl_wait();
    constexpr int ITEMS = D / 8;   // of a head
    const int r0 = blockIdx.x * READ_ROWS, most = live_rows(live, n), u = blockIdx.y * 256 + threadIdx.x;
    if (u >= 2 * c.Hkv * ITEMS) return;
    const int head = u / ITEMS, w0 = u % ITEMS;
    const bool is_k = head < c.Hkv;
    int slot[READ_ROWS];
    uint32_t w[READ_ROWS];
    uint16_t d[READ_ROWS];
#pragma unroll
    for (int i = 0; i < READ_ROWS; i++) slot[i] = r0 + i < most ? ld_prev(slots + r0 + i) : -1;
#pragma unroll
    for (int i = 0; i < READ_ROWS; i++) {
        const int page = slot[i] / c.page_tokens;
        if (slot[i] < 0 || page >= c.n_pages) {
            slot[i] = -1;
            continue;
        }
        const int in_page = slot[i] - page * c.page_tokens, i16 = in_page % GROUP;
        const uint8_t *g = group_at(c, page, is_k ? head : head - c.Hkv, in_page);
        if (is_k) {
            w[i] = ld_prev(reinterpret_cast<const uint32_t *>(g + k_word_at(D, i16, w0 / 4, w0 % 4)));
            d[i] = ld_prev(reinterpret_cast<const uint16_t *>(g + k_scale_at(D, i16, w0 / 4)));
        } else {
            const uint8_t *b = g + v_byte_at(D, i16, w0 / 2, w0 % 2 * 4);
            w[i] = ld_prev(b) | (uint32_t)ld_prev(b + 64) << 8 | (uint32_t)ld_prev(b + 128) << 16 | (uint32_t)ld_prev(b + 192) << 24;
            d[i] = ld_prev(reinterpret_cast<const uint16_t *>(g + v_scale_at(D, i16, w0 / 4)));
        }
    }
    const int x0 = is_k ? w0 / 4 * 32 + w0 % 4 * 4 : w0 / 2 * 16 + w0 % 2 * 4, x1 = x0 + (is_k ? 16 : 8);
#pragma unroll
    for (int i = 0; i < READ_ROWS; i++) {
        if (slot[i] < 0) continue;
        Y *row = out + (r0 + i) * out_stride + (int64_t)head * D;
        const float df = __half2float(__ushort_as_half(d[i]));
        store_row4(row + x0, code_values(w[i], df), wide);
        store_row4(row + x1, code_values(w[i] >> 4, df), wide);
    }
}

}  // namespace

qk_status launch_kv_append(const KvCache &c, int elem, const void *q, int64_t q_stride, int n_heads, const void *k,
                           int64_t k_stride, const void *v, int64_t v_stride, int T, const int32_t *slots,
                           const KvRope &rope, int q_elem, void *q_out, int64_t q_out_stride, const int32_t *live,
                           cudaStream_t s) {
    const bool wide = row_wide(k, k_stride, elem) && row_wide(v, v_stride, elem) && (n_heads == 0 || row_wide(q, q_stride, elem));
    const bool q_wide = row_wide(q_out, q_out_stride, q_elem);
    const auto go = [&](auto x, auto y) {
        using X = decltype(x);
        using Q = decltype(y);
        const bool halves = rope.kind == QK_ROPE_HALVES && rope.dims > 0;
        auto *kernel = halves ? (c.D == 64    ? kv_append_kernel<64, true, X, Q>
                                 : c.D == 128 ? kv_append_kernel<128, true, X, Q>
                                              : kv_append_kernel<256, true, X, Q>)
                              : (c.D == 64    ? kv_append_kernel<64, false, X, Q>
                                 : c.D == 128 ? kv_append_kernel<128, false, X, Q>
                                              : kv_append_kernel<256, false, X, Q>);
        return launch_pdl("kv_append", kernel, dim3((unsigned)T), dim3(256), 0, s, c, static_cast<const X *>(q), q_stride, n_heads,
                          static_cast<const X *>(k), k_stride, static_cast<const X *>(v), v_stride, T, slots, rope,
                          static_cast<Q *>(q_out), q_out_stride, wide, q_wide, live);
    };
    if (elem == QK_ELEM_F32) return q_elem == QK_ELEM_F32 ? go(float{}, float{}) : go(float{}, __nv_bfloat16{});
    return q_elem == QK_ELEM_F32 ? go(__nv_bfloat16{}, float{}) : go(__nv_bfloat16{}, __nv_bfloat16{});
}

qk_status launch_kv_read(const KvCache &c, const int32_t *slots, int n, int elem, void *out, int64_t out_stride,
                         const int32_t *live, cudaStream_t s) {
    const dim3 grid((unsigned)ceil_div(n, READ_ROWS), (unsigned)ceil_div(2 * c.Hkv * (c.D / 8), 256));
    const bool wide = row_wide(out, out_stride, elem);
    const auto go = [&](auto y) {
        using Y = decltype(y);
        auto *kernel = c.D == 64 ? kv_read_kernel<64, Y> : c.D == 128 ? kv_read_kernel<128, Y> : kv_read_kernel<256, Y>;
        return launch_pdl("kv_read", kernel, grid, dim3(256), 0, s, c, slots, n, static_cast<Y *>(out), out_stride, wide, live);
    };
    return elem == QK_ELEM_F32 ? go(float{}) : go(__nv_bfloat16{});
}

}  // namespace qk

// The 4-bit key/value cache: places inside a page (the layout is given in qk.h), rows of either element type.
#pragma once

#include <cuda_bf16.h>

#include "qk_internal.cuh"

namespace qk {

constexpr int GROUP = 16;   // tokens of a group

// Bytes of a group: codes of k (8 D), scales of k (D), codes of v (8 D), scales of v (D).
__host__ __device__ constexpr int group_bytes(int D) { return 18 * D; }

struct KvCache {
    uint8_t *pages;
    int n_pages, page_tokens, Hkv, D;
};
inline KvCache kv_cache(const qk_kv_cache *c) {
    return {static_cast<uint8_t *>(c->pages), (int)c->n_pages, c->page_tokens, c->n_kv_heads, c->head_dim};
}
// The group of token `in_page` of a page and head; the page is inside the cache.
__device__ __forceinline__ uint8_t *group_at(const KvCache &c, int page, int head, int in_page) {
    return c.pages + (((int64_t)page * c.Hkv + head) * (c.page_tokens / GROUP) + in_page / GROUP) * group_bytes(c.D);
}

// Places in a group of D columns: token i, block b (32 columns), word t of a block (columns 4t..4t+3 low, 16+4t.. high).
__device__ __forceinline__ int k_word_at(int D, int i, int b, int t) {
    const int W = D / 32 < 4 ? D / 32 : 4;
    return ((b / W * GROUP + i) * 4 + t) * 4 * W + b % W * 4;
}
__device__ __forceinline__ int k_scale_at(int D, int i, int b) { return 8 * D + 2 * (i * (D / 32) + b); }
// columns 16 m + g (low nibble) and 16 m + 8 + g (high)
__device__ __forceinline__ int v_byte_at(int D, int i, int m, int g) {
    return 9 * D + ((m / 4 * 8 + g) * 4 + i % 8 / 2) * 16 + m % 4 * 4 + 2 * (i % 2) + i / 8;
}
__device__ __forceinline__ int v_scale_at(int D, int i, int b) {
    return 17 * D + 2 * ((i % 8 / 2 * (D / 32) + b) * 4 + i % 2 + i / 8 * 2);
}

// Four consecutive elements of a row, as binary32. `wide`: the host has seen that every row starts where one load or
// store can take four elements (row_wide).
__device__ __forceinline__ float4 load_row4(const float *p, bool wide) {
    if (wide) return ld_prev(reinterpret_cast<const float4 *>(p));
    return make_float4(ld_prev(p), ld_prev(p + 1), ld_prev(p + 2), ld_prev(p + 3));
}
__device__ __forceinline__ uint2 load_bf16x4(const __nv_bfloat16 *p, bool wide) {
    const uint16_t *s = reinterpret_cast<const uint16_t *>(p);
    if (wide) return ld_prev(reinterpret_cast<const uint2 *>(p));
    return make_uint2(ld_prev(s) | (uint32_t)ld_prev(s + 1) << 16, ld_prev(s + 2) | (uint32_t)ld_prev(s + 3) << 16);
}
__device__ __forceinline__ float4 bf16x4(uint2 v) {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load_row4(const __nv_bfloat16 *p, bool wide) { return bf16x4(load_bf16x4(p, wide)); }
__device__ __forceinline__ void store_row4(float *p, float4 v, bool wide) {
    if (wide) {
        *reinterpret_cast<float4 *>(p) = v;
    } else {
        p[0] = v.x;
        p[1] = v.y;
        p[2] = v.z;
        p[3] = v.w;
    }
}
__device__ __forceinline__ void store_row4(__nv_bfloat16 *p, float4 v, bool wide) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    if (wide) {
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    } else {
        p[0] = lo.x;
        p[1] = lo.y;
        p[2] = hi.x;
        p[3] = hi.y;
    }
}
inline bool row_wide(const void *p, int64_t stride, int elem) {
    const int size = elem == QK_ELEM_F32 ? 4 : 2;
    return reinterpret_cast<uintptr_t>(p) % (4 * size) == 0 && stride % 4 == 0;
}

// Kernel launchers of the cache and its attention; arguments already validated.
struct KvRope {
    int kind, dims, n_axes;   // dims = 0: nothing is rotated
    const int32_t *positions;
    const float *freqs;
};
qk_status launch_kv_append(const KvCache &c, int elem, const void *q, int64_t q_stride, int n_heads, const void *k,
                           int64_t k_stride, const void *v, int64_t v_stride, int T, const int32_t *slots,
                           const KvRope &rope, int q_elem, void *q_out, int64_t q_out_stride, const int32_t *live,
                           cudaStream_t s);
qk_status launch_kv_read(const KvCache &c, const int32_t *slots, int n, int elem, void *out, int64_t out_stride,
                         const int32_t *live, cudaStream_t s);
qk_status launch_attn_decode(const KvCache &c, const qk_attn &a, int B, int T, uint8_t *img, int64_t row_blocks,
                             const int32_t *live, void *ws, cudaStream_t s);
qk_status read_attn_decode_faults(uint32_t *faults);
qk_status read_attn_wide_faults(uint32_t *faults);
qk_status read_attn_prefill_faults(uint32_t *faults);
int64_t attn_decode_workspace_bytes(int Hkv, int D, int n_heads, int64_t B, int T);
qk_status launch_attn_prefill(const KvCache &c, const qk_attn &a, int B, int rows, const int32_t *q_offsets, int max_kv,
                              int8_t *qs, uint16_t *d, int64_t row_blocks, const int32_t *live, void *ws, cudaStream_t s);
int64_t attn_prefill_workspace_bytes(int Hkv, int D, int64_t B, int64_t max_kv);

}  // namespace qk

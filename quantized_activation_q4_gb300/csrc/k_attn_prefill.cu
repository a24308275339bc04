// Attention of prompts and chunks of prompts over the 4-bit cache (qk_attn_prefill), on tcgen05.
//
// attn_stage_kernel turns the call's pages into binary16 once: keys [token][column] and values transposed
// [column][token], each (code - 8) * d rounded once and held to +-65504, so that both products read their second operand
// K-major by plain tensor copies. Inside a group of 16 the tokens are in the order of the value codes' words (position 4 t + s
// is token 2 t + s % 2 + 8 (s / 2)), in both, so that the words are unpacked without exchanges; the mask undoes it.
//
// attn_prefill_kernel: a CTA takes 128 rows (query token, head of the group) a tile, two tiles where the output fits
// (head_dim 64 and 128), of one sequence and key/value head, and walks over the keys that they see in steps of BN. For
// each tile S = Q K^T goes to tensor memory; two threads a row read a half each, keep the running maximum and sum, and write
// the weights back over it in binary16, the first operand of O += P V, which begins when the first half is there. While one
// tile's threads are at it, the tensor cores work on the other's products. O is rescaled only when a row's maximum grew by
// more than 2^8. Where tiles are fewer than the device has room for, their keys are shared out and attn_join_kernel adds up.
//
// Bound by the tensor cores and, nearly as much, by the chain scores - weights - products of a tile: at D = 128 a step of two
// tiles takes 3040 cycles, the products alone 2400 (2048 at their peak rate). 1024 rows of 28 heads over 4 behind 32000 keys:
// 314 us = 1.52 PFLOP/s (tensor pipe 68% active) and 35 for staging and join, 68% of the measured bf16 rate in all; 3325 rows
// without a past: 91 us and 7. What the steps gave there (us): one thread a row 127, two 97; products issued under
// elect.sync and not by lane 0 176 -> 127; rescaling eight columns at a time 228 -> 97 (with 32 the scores spilled).

#include <algorithm>

#include "qk_kv.cuh"
#include "qk_tc.cuh"

namespace qk {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E = 1.4426950408889634f;
constexpr int ROWS = 128;           // rows of a tile: lanes of tensor memory
constexpr int PAD = 128;            // staged lengths are whole multiples
constexpr float HEADROOM = 8.0f;    // the reference maximum moves when a logit is 2^8 above it
constexpr float LIFT = 6.0f;        // weights are held times 2^6 below the reference: at most 2^14
constexpr float UNLIFT = 0x1p-6f;

struct PrefillArgs {
    CUtensorMap kmap, vmap;   // keys [B Hkv Lpad][D], values [B Hkv D][Lpad]
    KvCache c;
    qk_attn a;
    int B, rows, G, max_kv, lpad;
    const int32_t *offsets, *live;
    __half *k, *v;
    uint8_t *there;           // [B][lpad / 16] whether a group's page exists
    int8_t *qs;
    uint16_t *d;
    int64_t row_blocks;
    bool q_wide, out_wide, out16;   // out16: bfloat16 rows start on 16-byte boundaries
    // a tile's keys in `parts` shares of steps; with more than one, unnormalised outputs [CTA][row][D] and, for each
    // row, its reference (minus infinity: no key) and the sum of the weights relative to it
    int parts;
    float *part_o;
    float2 *part_ml;
};

// Rows and keys of a sequence.
struct Span1 {
    int first, n, len, seen, base;   // first row, rows, keys, first key that any row sees, that one rounded down to 128
};
__device__ __forceinline__ Span1 span_of(const PrefillArgs &p, int b) {
    Span1 s;
    s.first = min(max(ld_prev(p.offsets + b), 0), p.rows);
    s.n = max(0, min(max(ld_prev(p.offsets + b + 1), 0), p.rows) - s.first);
    s.len = min(max(ld_prev(p.a.kv_lens + b), 0), p.max_kv);
    s.seen = p.a.window > 0 ? max(0, s.len - s.n + 1 - p.a.window) : 0;
    s.base = s.seen & ~(PAD - 1);
    return s;
}

// The tile of rows that a CTA takes: tiles are counted from the last sequence's last (a causal tile sees the more keys the
// later it is, and the long ones go first). One warp looks; .x < 0: there are not so many.
__device__ __forceinline__ int2 find_tile(const PrefillArgs &p, int64_t skip, int cta_rows) {
    const int live = live_rows(p.live, p.B), lane = threadIdx.x & 31;
    for (int hi = live; hi > 0; hi -= 32) {
        const int b = hi - 1 - lane;
        const int64_t n = b >= 0 ? ((int64_t)span_of(p, b).n * p.G + cta_rows - 1) / cta_rows : 0;
        int64_t x = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t y = __shfl_up_sync(FULL, x, m);
            if (lane >= m) x += y;
        }
        const uint32_t mine = __ballot_sync(FULL, skip < x && skip >= x - n);
        if (mine) {
            const int at = __ffs(mine) - 1, tile = (int)(n - 1 - (skip - (x - n)));
            return make_int2(hi - 1 - at, __shfl_sync(FULL, tile, at));
        }
        skip -= __shfl_sync(FULL, x, 31);
    }
    return make_int2(-1, 0);
}

// ---------------------------------------------------------------- staging
// (code - 8) * d, at most binary16's largest value: an infinity would reach rows that do not see its key, as weight 0 times
// infinity.
__device__ __forceinline__ uint32_t value2(uint32_t v, uint32_t bias, __half2 d) {
    const __half2 most = half2_bits(0x7bff7bffu), x = __hmul2(__hsub2(half2_bits(v), half2_bits(bias)), d);
    const __half2 r = __hmax2(__hmin2(x, most), __hneg2(most));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t lo_half(uint32_t w) { return (w & 0x000F000Fu) | 0x64006400u; }   // 1024 + code
__device__ __forceinline__ uint32_t hi_half(uint32_t w) { return (w & 0x00F000F0u) | 0x54005400u; }   // 64 + code
constexpr uint32_t LO_BIAS = 0x64086408u, HI_BIAS = 0x54805480u;

// CTA (x, head, b): 64 tokens of a head. A warp takes a group; a lane takes words (block, t) of k and (column tile, t) of v.
template <int D>
__global__ void __launch_bounds__(128) attn_stage_kernel(const __grid_constant__ PrefillArgs p) {
    constexpr int NB = D / 32, W = NB < 4 ? NB : 4;
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
    const int token = (blockIdx.x * 4 + (threadIdx.x >> 5)) * GROUP;
    if (b >= live_rows(p.live, p.B)) return;
    const Span1 s = span_of(p, b);
    if (s.n == 0 || token < s.base || token >= (s.len + PAD - 1) / PAD * PAD) return;
    int page = -1;
    if (token < s.len) page = ld_prev(p.a.page_table + b * p.a.table_stride + token / p.c.page_tokens);
    const bool good = page >= 0 && page < p.c.n_pages;
    if (h == 0 && lane == 0) p.there[(int64_t)b * (p.lpad / GROUP) + token / GROUP] = good;
    const uint8_t *g = good ? group_at(p.c, page, h, token % p.c.page_tokens) : nullptr;
    const int64_t seg = (int64_t)b * p.c.Hkv + h;
    __half *k = p.k + (seg * p.lpad + token) * D, *v = p.v + seg * D * p.lpad + token;
    // keys: token i goes to position 4 (i % 8 / 2) + i % 2 + i / 8 * 2
#pragma unroll
    for (int x = lane; x < GROUP * 4 * (NB / W); x += 32) {
        const int t = x & 3, i = x / 4 % GROUP, bq = x / (4 * GROUP);
        const int row = 4 * (i % 8 / 2) + i % 2 + i / 8 * 2;
        const bool keep = good && token + i < s.len && token + i >= s.seen;
        uint32_t words[W], scales[W / 2];   // of W blocks side by side
        if (keep) {
            const uint8_t *kw = g + k_word_at(D, i, bq * W, t), *ks = g + k_scale_at(D, i, bq * W);
            if constexpr (W == 4) {
                const uint4 a = ld_prev(reinterpret_cast<const uint4 *>(kw));
                const uint2 d = ld_prev(reinterpret_cast<const uint2 *>(ks));
                words[0] = a.x, words[1] = a.y, words[2] = a.z, words[3] = a.w, scales[0] = d.x, scales[1] = d.y;
            } else {
                const uint2 a = ld_prev(reinterpret_cast<const uint2 *>(kw));
                words[0] = a.x, words[1] = a.y, scales[0] = ld_prev(reinterpret_cast<const uint32_t *>(ks));
            }
        }
#pragma unroll
        for (int e = 0; e < W; e++) {
            const int blk = bq * W + e;
            uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
            if (keep) {
                const uint32_t w = words[e], w8 = w >> 8;
                const __half2 ds = half2_bits(scales[e / 2]), d2 = e & 1 ? __high2half2(ds) : __low2half2(ds);
                const uint32_t a = value2(lo_half(w), LO_BIAS, d2), c = value2(lo_half(w8), LO_BIAS, d2);   // 0 2, 1 3
                const uint32_t y = value2(hi_half(w), HI_BIAS, d2), z = value2(hi_half(w8), HI_BIAS, d2);
                lo = make_uint2(__byte_perm(a, c, 0x5410), __byte_perm(a, c, 0x7632));
                hi = make_uint2(__byte_perm(y, z, 0x5410), __byte_perm(y, z, 0x7632));
            }
            __half *to = k + row * D + 32 * blk + 4 * t;
            *reinterpret_cast<uint2 *>(to) = lo;
            *reinterpret_cast<uint2 *>(to + 16) = hi;
        }
    }
    // values: a word holds the tokens of positions 4 t .. 4 t + 3 of columns 16 m + u and 16 m + 8 + u
#pragma unroll
    for (int x = lane; x < D / 64 * 32; x += 32) {
        const int t = x & 3, u = x / 4 % 8, mq = x / 32;
        const auto seen = [&](int j) { return j >= s.seen && j < s.len; };
        const bool k0 = seen(token + 2 * t), k1 = seen(token + 2 * t + 1), k2 = seen(token + 2 * t + 8), k3 = seen(token + 2 * t + 9);
        uint4 w = make_uint4(0, 0, 0, 0), d4 = w;   // two blocks' scales
        if (good) {
            w = ld_prev(reinterpret_cast<const uint4 *>(g + 9 * D + x * 16));
            d4 = ld_prev(reinterpret_cast<const uint4 *>(g + 17 * D + (t * NB + 2 * mq) * 8));
        }
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int m = mq * 4 + e;
            uint2 d = e < 2 ? make_uint2(d4.x, d4.y) : make_uint2(d4.z, d4.w);
            // (a scale behind the last key or in front of the first that is seen may be anything: it is taken as 0)
            d.x &= (k0 ? 0xffffu : 0) | (k1 ? 0xffff0000u : 0);
            d.y &= (k2 ? 0xffffu : 0) | (k3 ? 0xffff0000u : 0);
            const uint32_t y = words[e], y8 = y >> 8;
            __half *to = v + (int64_t)(16 * m + u) * p.lpad + 4 * t;
            *reinterpret_cast<uint2 *>(to) =
                make_uint2(value2(lo_half(y), LO_BIAS, half2_bits(d.x)), value2(lo_half(y8), LO_BIAS, half2_bits(d.y)));
            *reinterpret_cast<uint2 *>(to + (int64_t)8 * p.lpad) =
                make_uint2(value2(hi_half(y), HI_BIAS, half2_bits(d.x)), value2(hi_half(y8), HI_BIAS, half2_bits(d.y)));
        }
    }
}

// Logits (times log2 e) far from 0. A score is off by 2^-11 of its terms (its operands are binary16), so beyond 2^22 which of
// nearly equal logits is the larger is not known, and one number holds neither such a reference with the lift of the weights
// nor a score's product with the row's factor to a unit. While a row's reference is beyond, its factor is less by the power
// of two that brings the reference below: logits within about 2^-18 of it share the weight, all others get none.
__device__ __forceinline__ float far_factor(float reference) {
    const int e = (int)(__float_as_uint(reference) >> 23 & 255) - (127 + 21);
    return e > 0 && reference != -INFINITY ? __uint_as_float((uint32_t)(127 - e) << 23) : 1.0f;
}
// a / b of numbers that differ by a power of two alone
__device__ __forceinline__ float power_ratio(float a, float b) {
    return __uint_as_float(0x3f800000u + __float_as_uint(a) - __float_as_uint(b));
}

// ---------------------------------------------------------------- attention
// Products with K-major operands in shared memory, 128-byte swizzle (sdesc): the descriptors' low words plus a constant,
// put together where they are used (held ready as 64-bit words they cost the kernel its registers).
__device__ __forceinline__ uint32_t sdesc_low(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
constexpr uint32_t SDESC_HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);
template <int A, int B>   // D (tensor memory) (+)= A (shared memory) x B (shared memory), A and B bytes further on
__device__ __forceinline__ void mma_ss(uint32_t tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b32 x, y;\n .reg .b64 da, db;\n setp.ne.u32 p, %4, 0;\n"
        " add.u32 x, %1, %5;\n add.u32 y, %2, %6;\n mov.b64 da, {x, %7};\n mov.b64 db, {y, %7};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(A >> 4), "n"(B >> 4), "n"(SDESC_HIGH)
        : "memory");
}
template <int A, int B>   // the same with A in tensor memory, A columns further on
__device__ __forceinline__ void mma_ts(uint32_t tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b32 x, y;\n .reg .b64 db;\n setp.ne.u32 p, %4, 0;\n"
        " add.u32 x, %1, %5;\n add.u32 y, %2, %6;\n mov.b64 db, {y, %7};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n}\n" ::"r"(tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(A), "n"(B >> 4), "n"(SDESC_HIGH)
        : "memory");
}
// K = 16 * N of S = Q K^T from step KS on; of O += P V
template <int D, int BN, int KS, int N>
__device__ __forceinline__ void mma_scores(uint32_t tmem, uint32_t q, uint32_t k) {
    if constexpr (N > 0) {
        mma_ss<(KS >> 2) * ROWS * 128 + 32 * (KS & 3), (KS >> 2) * BN * 128 + 32 * (KS & 3)>(tmem, q, k, mma_idesc(BN), KS != 0);
        mma_scores<D, BN, KS + 1, N - 1>(tmem, q, k);
    }
}
template <int D, int KS, int N>
__device__ __forceinline__ void mma_outputs(uint32_t tmem, uint32_t p, uint32_t v, uint32_t accumulate) {
    if constexpr (N > 0) {
        mma_ts<8 * KS, (KS >> 2) * D * 128 + 32 * (KS & 3)>(tmem, p, v, mma_idesc(D), accumulate);
        mma_outputs<D, KS + 1, N - 1>(tmem, p, v, 1);
    }
}
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(a));
}
__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t *v) {   // waits
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n tcgen05.wait::ld.sync.aligned;"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// (the loaded registers pass through, so that no use of them moves up)
__device__ __forceinline__ void tmem_wait_ld(uint32_t *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                   "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Eight elements of a row, as loaded.
template <typename Q>
struct Row8 {
    float4 a, b;
    __device__ __forceinline__ void clear() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void load(const float *p, bool wide) {
        a = load_row4(p, wide);
        b = load_row4(p + 4, wide);
    }
    __device__ __forceinline__ float4 low() const { return a; }
    __device__ __forceinline__ float4 high() const { return b; }
};
template <>
struct Row8<__nv_bfloat16> {
    uint2 a, b;
    __device__ __forceinline__ void clear() { a = b = make_uint2(0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool wide) {
        a = load_bf16x4(p, wide);
        b = load_bf16x4(p + 4, wide);
    }
    __device__ __forceinline__ float4 low() const { return bf16x4(a); }
    __device__ __forceinline__ float4 high() const { return bf16x4(b); }
};
// 16 rows of a tile's queries, from row `row` on: binary16 of q / 2^e with 2^e above the row's largest magnitude, and what
// the scores are multiplied with, scale * log2 e * 2^e. `first`: the sequence's first row, `rho`: the tile's first of its
// rows_all rows (token, head).
template <int D, typename Q>
__device__ __forceinline__ void load_queries(const PrefillArgs &p, const Q *q, int first, int h, int rho, int rows_all,
                                             int row, uint8_t *tile, float *factor) {
    constexpr int LANES = D / 8, TURN = 32 / LANES;   // of a row; rows of a turn
    const int lane = threadIdx.x & 31, unit = lane % LANES;
    constexpr int AHEAD = (sizeof(Q) == 2 ? 8 : 4) < 16 / TURN ? (sizeof(Q) == 2 ? 8 : 4) : 16 / TURN;   // turns loaded together
#pragma unroll 1
    for (int x0 = 0; x0 < 16; x0 += TURN * AHEAD) {
        Row8<Q> v[AHEAD];
#pragma unroll
        for (int x = 0; x < AHEAD; x++) {
            const int r = rho + row + x0 + x * TURN + lane / LANES;
            v[x].clear();
            if (r < rows_all) {
                const int token = r / p.G, head = h * p.G + r - token * p.G;
                v[x].load(q + (int64_t)(first + token) * p.a.q_stride + (int64_t)head * D + 8 * unit, p.q_wide);
            }
        }
#pragma unroll
        for (int x = 0; x < AHEAD; x++) {
            const int r = row + x0 + x * TURN + lane / LANES;
            const float4 a = v[x].low(), c = v[x].high();
            float top = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                              fmaxf(fmaxf(fabsf(c.x), fabsf(c.y)), fmaxf(fabsf(c.z), fabsf(c.w))));
#pragma unroll
            for (int m = 1; m < LANES; m <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, m));
            // (2^e and its inverse are normal numbers: from 2^126 on it is above a quarter of the magnitude)
            const int e = min(max((int)(__float_as_uint(top) >> 23) - 126, -126), 126);
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
            if (unit == 0) factor[r] = fmaxf(p.a.scale * __uint_as_float((uint32_t)(127 + e) << 23) * LOG2E, 0x1p-126f);
            *reinterpret_cast<uint4 *>(tile + (unit / 8) * ROWS * 128 + r * 128 + (((unit & 7) ^ (r & 7)) << 4)) =
                make_uint4(pack2(a.x * down, a.y * down), pack2(a.z * down, a.w * down), pack2(c.x * down, c.y * down),
                           pack2(c.z * down, c.w * down));
        }
    }
}

// A warp's 32 rows of W bytes, put into shared memory a row a lane, to global memory: 16 bytes a lane, whole rows a store.
// A row's unit c is at c ^ (row % units) so that neither side meets bank conflicts. base + off: the lane's own row.
template <int CH>
__device__ __forceinline__ uint8_t *staged(uint8_t *rows, int row, int c) {
    return rows + row * CH + ((c ^ (row % (CH / 16))) << 4);
}
template <int CH, int W>
__device__ __forceinline__ void store_rows(uint8_t *rows, uint8_t *base, int64_t off, bool there) {
    constexpr int LANES = W / 16;
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll 4
    for (int r0 = 0; r0 < 32; r0 += 32 / LANES) {
        const int r = r0 + lane / LANES, c = lane % LANES;
        const uint4 v = *reinterpret_cast<const uint4 *>(staged<CH>(rows, r, c));
        const int64_t o = __shfl_sync(FULL, off, r);
        if (__shfl_sync(FULL, (int)there, r)) *reinterpret_cast<uint4 *>(base + o + 16 * c) = v;
    }
    __syncwarp();
}

template <int D>
struct Shape {
    static constexpr int TILES = D == 256 ? 1 : 2;       // row tiles of a CTA
    static constexpr int BN = D == 256 ? 64 : 128;       // keys of a step
    static constexpr int STAGES = 2;
    static constexpr int Q_BYTES = ROWS * D * 2;         // one tile; chunks of 64 columns, 16 KB each
    static constexpr int K_BYTES = BN * D * 2;
    static constexpr int V_BYTES = D * BN * 2;
    static constexpr int O_TMEM = 256;                   // S (then P) of tile i at 128 i, O at 256 + D i
    static constexpr int OFF_K = TILES * Q_BYTES;
    static constexpr int OFF_V = OFF_K + STAGES * K_BYTES;
    static constexpr int OFF_SCALE = OFF_V + STAGES * V_BYTES;   // a row's factor
    static constexpr int OFF_TOP = OFF_SCALE + TILES * ROWS * 4;   // a thread's maxima of two steps, and its row's factor
    static constexpr int OFF_BAR = OFF_TOP + TILES * 2 * 3 * ROWS * 4;
    // q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], done
    static constexpr int N_BARS = 1 + 4 * STAGES + 4 * 2 + 1;
    static constexpr int SMEM = OFF_BAR + 8 * N_BARS + 16 + 1024;
    static constexpr int THREADS = (8 * TILES + 2) * 32;   // two threads a row, a warp for copies, one for products
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(O_TMEM + TILES * D <= 512, "tensor memory");
};

template <int D>
__global__ void __launch_bounds__(Shape<D>::THREADS, 1) attn_prefill_kernel(const __grid_constant__ PrefillArgs p) {
    using Z = Shape<D>;
    constexpr int BN = Z::BN, TILES = Z::TILES, NB = D / 32;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int2 where;   // sequence, tile in it
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t q_full = sbase + Z::OFF_BAR, k_full = q_full + 8, k_empty = k_full + 16, v_full = k_empty + 16,
                   v_empty = v_full + 16, s_full = v_empty + 16, p_half = s_full + 16, p_full = p_half + 16,
                   o_full = p_full + 16, done = o_full + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Z::OFF_BAR + 8 * Z::N_BARS);
    float *factor = reinterpret_cast<float *>(smem + Z::OFF_SCALE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int TMA_WARP = 8 * TILES, MMA_WARP = TMA_WARP + 1, HALF = BN / 2;

    if (threadIdx.x == 0) {
        mbar_init(q_full, TILES * 2 * ROWS);
        for (int s = 0; s < 2; s++) {
            mbar_init(k_full + 8 * s, 1);
            mbar_init(k_empty + 8 * s, 1);
            mbar_init(v_full + 8 * s, 1);
            mbar_init(v_empty + 8 * s, 1);
            mbar_init(s_full + 8 * s, 1);
            mbar_init(p_half + 8 * s, ROWS);   // the weights of a step's first and second half
            mbar_init(p_full + 8 * s, ROWS);
            mbar_init(o_full + 8 * s, 1);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_trigger();
    pdl_wait();
    const int part = blockIdx.x % p.parts, h = blockIdx.x / p.parts % p.c.Hkv;
    constexpr int CTA_ROWS = TILES * ROWS;
    if (warp == 0) {
        const int2 w = find_tile(p, blockIdx.x / p.parts / p.c.Hkv, CTA_ROWS);
        if (lane == 0) where = w;
    }
    __syncthreads();
    const int b = where.x;
    if (b < 0) return;
    const Span1 sq = span_of(p, b);
    const int rows_all = sq.n * p.G, row0 = where.y * CTA_ROWS;   // of the sequence's n * G rows
    const int row_last = min(row0 + CTA_ROWS, rows_all) - 1;
    // keys that any of the rows sees, from a step's beginning
    const int end = sq.len - sq.n + row_last / p.G + 1;
    int begin = 0;
    if (p.a.window > 0) begin = max(0, sq.len - sq.n + row0 / p.G + 1 - p.a.window) / BN * BN;
    int steps = end > begin ? (end - begin + BN - 1) / BN : 0;
    if (p.parts > 1) {
        const int from = (int)((int64_t)steps * part / p.parts), to = (int)((int64_t)steps * (part + 1) / p.parts);
        begin += from * BN;
        steps = to - from;
    }

    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int64_t seg = (int64_t)b * p.c.Hkv + h;

    if (warp == TMA_WARP) {   // ---------------- copies
        if (elect_one()) {
            int j = 0;
            for (; j < steps; j++) {
                const uint32_t s = j % 2, par = (j / 2 - 1) & 1u;
                const int kv = begin + j * BN;
                if (j >= 2 && !mbar_wait(k_empty + 8 * s, par)) break;
                mbar_expect_tx(k_full + 8 * s, Z::K_BYTES);
                for (int x = 0; x < D / 64; x++)
                    tma_2d(sbase + Z::OFF_K + s * Z::K_BYTES + x * BN * 128, &p.kmap, 64 * x, (int)(seg * p.lpad) + kv,
                           k_full + 8 * s);
                if (j >= 2 && !mbar_wait(v_empty + 8 * s, par)) {
                    mbar_wait(k_full + 8 * s, (j / 2) & 1u);
                    break;
                }
                mbar_expect_tx(v_full + 8 * s, Z::V_BYTES);
                for (int x = 0; x < BN / 64; x++)
                    tma_2d(sbase + Z::OFF_V + s * Z::V_BYTES + x * D * 128, &p.vmap, kv + 64 * x, (int)(seg * D),
                           v_full + 8 * s);
            }
            // every copy has landed before the CTA can go, also after a wait ran out
            for (int x = j > 2 ? j - 2 : 0; x < j; x++)
                if (!mbar_wait(k_full + 8 * (x % 2), (x / 2) & 1u) || !mbar_wait(v_full + 8 * (x % 2), (x / 2) & 1u)) break;
        }
    } else if (warp == MMA_WARP) {   // ---------------- products
        if (elect_one()) {
            bool ok = steps > 0 && mbar_wait(q_full, 0);
            const uint32_t q0 = sdesc_low(sbase), k0 = sdesc_low(sbase + Z::OFF_K), v0 = sdesc_low(sbase + Z::OFF_V);
            const auto scores = [&](int i, int j) {   // S of tile i, step j
                mma_scores<D, BN, 0, D / 16>(tmem + 128 * i, q0 + i * (Z::Q_BYTES >> 4), k0 + (j % 2) * (Z::K_BYTES >> 4));
                tc_commit(s_full + 8 * i);
            };
            if (ok) {
                tc_fence_after();
                ok = mbar_wait(k_full, 0);
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < TILES; i++) scores(i, 0);
                    tc_commit(k_empty);
                }
            }
            for (int j = 0; j < steps && ok; j++) {
                ok = mbar_wait(v_full + 8 * (j % 2), (j / 2) & 1u);
                if (ok && j + 1 < steps) ok = mbar_wait(k_full + 8 * ((j + 1) % 2), ((j + 1) / 2) & 1u);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < TILES; i++) {
                    if (ok) ok = mbar_wait(p_half + 8 * i, j & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    mma_outputs<D, 0, BN / 32>(tmem + Z::O_TMEM + D * i, tmem + 128 * i, v0 + (j % 2) * (Z::V_BYTES >> 4), j != 0);
                    ok = mbar_wait(p_full + 8 * i, j & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    mma_outputs<D, BN / 32, BN / 32>(tmem + Z::O_TMEM + D * i, tmem + 128 * i, v0 + (j % 2) * (Z::V_BYTES >> 4), 1);
                    if (j + 1 < steps)
                        scores(i, j + 1);
                    else
                        tc_commit(o_full + 8 * i);
                }
                if (!ok) break;
                tc_commit(v_empty + 8 * (j % 2));
                if (j + 1 < steps) tc_commit(k_empty + 8 * ((j + 1) % 2));
            }
            tc_commit(done);   // no product is under way when the tensor memory is freed
            mbar_wait(done, 0);
        }
    } else if (warp < TMA_WARP) {   // ---------------- two threads a row, a half of a step's keys each
        const int i = warp / 8, quad = warp & 3, hf = warp / 4 % 2, r = 32 * quad + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        const uint32_t st = lanes + 128 * i, ot = lanes + Z::O_TMEM + D * i;
        // queries: eight columns a lane, so that a load takes whole rows; a row's power of two taken out; in the layout of a
        // K-major operand
        if (steps > 0) {
            if (p.a.q_elem == QK_ELEM_F32)
                load_queries<D>(p, static_cast<const float *>(p.a.q), sq.first, h, row0 + i * ROWS, rows_all, 32 * quad + 16 * hf,
                                smem + i * Z::Q_BYTES, factor + i * ROWS);
            else
                load_queries<D>(p, static_cast<const __nv_bfloat16 *>(p.a.q), sq.first, h, row0 + i * ROWS, rows_all,
                                32 * quad + 16 * hf, smem + i * Z::Q_BYTES, factor + i * ROWS);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(q_full);
        }
        // the two warps of 32 rows meet (what one reads of tensor memory and the other writes are these rows' lanes)
        const auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + 4 * i + quad) : "memory"); };
        meet();   // the factors are written
        float *const mine = reinterpret_cast<float *>(smem + Z::OFF_TOP) + (i * 2 + hf) * 3 * ROWS + r;
        const float *const other = reinterpret_cast<float *>(smem + Z::OFF_TOP) + (i * 2 + 1 - hf) * 3 * ROWS + r;
        const int rho = row0 + i * ROWS + r;
        const bool there = rho < rows_all;
        const int token = there ? rho / p.G : sq.n - 1, head = h * p.G + (there ? rho - token * p.G : 0);
        const int my_end = sq.len - sq.n + token + 1, my_begin = p.a.window > 0 ? max(0, my_end - p.a.window) : 0;
        mine[2 * ROWS] = steps > 0 ? factor[i * ROWS + r] : 1.0f;
        float c = mine[2 * ROWS], ref = -INFINITY, off = 0.0f, sum = 0.0f;   // c: the factor, or less by far_factor
        bool ok = true;
        for (int j = 0; j < steps; j++) {   // (a wait that ran out goes on without work: both halves meet in every step)
            const int kv = begin + j * BN + hf * HALF;
            if (ok) ok = __all_sync(FULL, mbar_wait(s_full + 8 * i, j & 1u));
            tc_fence_after();
            uint32_t sv[HALF];
            // whether the pages of the keys exist, a byte a group
            const uint8_t *there16 = p.there + (int64_t)b * (p.lpad / GROUP) + kv / GROUP;
            const uint32_t exist = HALF == 64 ? ld_prev(reinterpret_cast<const uint32_t *>(there16))
                                              : ld_prev(reinterpret_cast<const uint16_t *>(there16)) | 0x01010000u;
#pragma unroll
            for (int x = 0; x < HALF; x += 32) tmem_ld32(st + hf * HALF + x, sv + x);
#pragma unroll
            for (int x = 0; x < HALF; x += 32) tmem_wait_ld(sv + x);
            const bool hidden = kv + HALF > my_end || kv < my_begin || exist != 0x01010101u;
            if (__any_sync(FULL, hidden)) {
#pragma unroll
                for (int x = 0; x < HALF; x++) {
                    const int key = kv + x / 16 * 16 + x % 16 / 4 * 2 + x % 2 + x % 4 / 2 * 8;
                    if (key >= my_end || key < my_begin || !(exist >> (8 * (x / 16)) & 1)) sv[x] = 0xff800000u;
                }
            }
            float tops[8];
#pragma unroll
            for (int x = 0; x < 8; x++) tops[x] = __uint_as_float(sv[x]);
#pragma unroll
            for (int x = 8; x < HALF; x += 16)
#pragma unroll
                for (int y = 0; y < 8; y++)
                    tops[y] = x + 8 < HALF ? fmaxf(fmaxf(tops[y], __uint_as_float(sv[x + y])), __uint_as_float(sv[x + 8 + y]))
                                           : fmaxf(tops[y], __uint_as_float(sv[x + y]));
            float top = fmaxf(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])),
                              fmaxf(fmaxf(tops[4], tops[5]), fmaxf(tops[6], tops[7])));
            // the other half's maximum (where the weights go, the scores of both halves have been read)
            mine[(j & 1) * ROWS] = top;
            tc_fence_before();
            meet();
            tc_fence_after();
            top = fmaxf(top, other[(j & 1) * ROWS]);
            top = top == -INFINITY ? top : top * c;
            const bool move = top - ref > HEADROOM;
            if (__any_sync(FULL, move)) {
                const float now = move ? top : ref;
                const float down = ref == -INFINITY ? 0.0f : ex2(ref - now);
                // the step before has been added: its products came before these scores. The first half's thread takes
                // the whole row, since its weights start the next products
                if (j > 0 && hf == 0) {
#pragma unroll 1
                    for (int x = 0; x < D; x += 8) {   // (few columns at once: the scores stay in registers)
                        uint32_t v[8];
                        tmem_ld8(ot + x, v);
#pragma unroll
                        for (int y = 0; y < 8; y++) v[y] = __float_as_uint(__uint_as_float(v[y]) * down);
                        tmem_st8(ot + x, v);
                    }
                }
                sum *= down;
                const float c0 = mine[2 * ROWS], logit = now * power_ratio(c0, c), f = far_factor(logit);
                c = c0 * f;
                ref = logit * f;
                off = ref == -INFINITY ? 0.0f : ref - LIFT;
            }
            uint64_t sums[2] = {0, 0};
            const uint64_t c2 = two(c, c), off2 = two(-off, -off);
#pragma unroll
            for (int x0 = 0; x0 < HALF; x0 += 16) {
                uint32_t w[8];
#pragma unroll
                for (int x = 0; x < 16; x += 2) {
                    const float2 e = apart(fma2(two(__uint_as_float(sv[x0 + x]), __uint_as_float(sv[x0 + x + 1])), c2, off2));
                    const float p0 = ex2(e.x), p1 = ex2(e.y);
                    sums[x / 2 % 2] = add2(sums[x / 2 % 2], two(p0, p1));
                    w[x / 2] = pack2(p0, p1);
                }
                tmem_st8(st + hf * (HALF / 2) + x0 / 2, w);
            }
            const float2 all = apart(add2(sums[0], sums[1]));
            sum += all.x + all.y;
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive((hf ? p_full : p_half) + 8 * i);
        }
        ref *= power_ratio(mine[2 * ROWS], c);
        // the row's sum, then its outputs: a half of the columns each
        mine[(steps & 1) * ROWS] = sum;
        meet();
        sum += other[(steps & 1) * ROWS];
        if (ok && steps > 0) ok = __all_sync(FULL, mbar_wait(o_full + 8 * i, 0));
        tc_fence_after();
        // Rows go through the shared memory of the tile's queries, which no product reads any more: D bytes a row for each warp,
        // half a head in bfloat16 or codes, a quarter of one in binary32.
        constexpr int CH = D;
        uint8_t *const rows = smem + i * Z::Q_BYTES + (warp & 7) * 32 * CH;
        const auto store_block = [&](const float (&y)[32], uint8_t *base, int64_t off, bool mine) {   // binary32
            constexpr int PIECE = CH < 128 ? 16 : 32;   // (at D = 64 a row has 64 bytes)
#pragma unroll
            for (int x0 = 0; x0 < 32; x0 += PIECE) {
#pragma unroll
                for (int x = 0; x < PIECE; x += 4)
                    *reinterpret_cast<float4 *>(staged<CH>(rows, lane, x / 4)) =
                        make_float4(y[x0 + x], y[x0 + x + 1], y[x0 + x + 2], y[x0 + x + 3]);
                store_rows<CH, PIECE * 4>(rows, base, off + x0 * 4, mine);
            }
        };
        if (p.parts > 1) {   // what this share of the keys gives; attn_join_kernel goes on
            const int64_t at = (int64_t)blockIdx.x * CTA_ROWS + i * ROWS + r;
            if (hf == 0 && there && ok) p.part_ml[at] = make_float2(ref, sum * UNLIFT);
#pragma unroll 1
            for (int k = hf * NB / 2; k < (hf + 1) * NB / 2 && steps > 0; k++) {
                uint32_t v[32];
                tmem_ld32(ot + 32 * k, v);
                tmem_wait_ld(v);
                float y[32];
#pragma unroll
                for (int x = 0; x < 32; x++) y[x] = __uint_as_float(v[x]) * UNLIFT;
                store_block(y, reinterpret_cast<uint8_t *>(p.part_o), (at * D + 32 * k) * 4, there && ok);
            }
        } else {
            float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // no key: 0
            if (p.a.sinks) {
                const float sink = ld_prev(p.a.sinks + head) * LOG2E;
                // relative to the larger of reference and sink: one far above the other takes all
                const float lead = fmaxf(sink, ref), down = ref == -INFINITY ? 0.0f : ex2(ref - lead) * UNLIFT;
                const float total = sink == -INFINITY ? sum * down : fmaf(sum, down, ex2(sink - lead));
                inv = total == 0.0f ? 0.0f : down / total;   // (a NaN row has no reference: its sum stays NaN)
            }
            const int64_t row = sq.first + token;
            const bool any = steps > 0 && inv != 0.0f, mine_ok = there && ok;
            const int k0 = hf * NB / 2;
            const auto block_of = [&](int k, float (&y)[32]) {
                if (steps > 0) {
                    uint32_t v[32];
                    tmem_ld32(ot + 32 * k, v);
                    tmem_wait_ld(v);
#pragma unroll
                    for (int x = 0; x < 32; x++) y[x] = any ? __uint_as_float(v[x]) * inv : 0.0f;
                } else {
#pragma unroll
                    for (int x = 0; x < 32; x++) y[x] = 0.0f;
                }
            };
            const int64_t at = row * p.a.out_stride + (int64_t)head * D + 32 * k0;
            if (p.a.out && p.a.out_elem == QK_ELEM_BF16) {
                uint16_t *const out = static_cast<uint16_t *>(p.a.out);
#pragma unroll 1
                for (int k = 0; k < NB / 2; k++) {
                    float y[32];
                    block_of(k0 + k, y);
#pragma unroll
                    for (int x = 0; x < 32; x += 8) {
                        const uint4 w = make_uint4(bf16x2(y[x], y[x + 1]), bf16x2(y[x + 2], y[x + 3]), bf16x2(y[x + 4], y[x + 5]),
                                                   bf16x2(y[x + 6], y[x + 7]));
                        if (p.out16) {
                            *reinterpret_cast<uint4 *>(staged<CH>(rows, lane, 4 * k + x / 8)) = w;
                        } else if (mine_ok) {
                            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int e = 0; e < 8; e++) out[at + 32 * k + x + e] = (uint16_t)(words[e / 2] >> (16 * (e & 1)));
                        }
                    }
                    __syncwarp();   // whole warps load from tensor memory
                }
                if (p.out16) store_rows<CH, CH>(rows, static_cast<uint8_t *>(p.a.out), at * 2, mine_ok);
            } else if (p.a.out) {
#pragma unroll 1
                for (int k = 0; k < NB / 2; k++) {
                    float y[32];
                    block_of(k0 + k, y);
                    float *const out = static_cast<float *>(p.a.out) + at + 32 * k;
                    if (p.out_wide) {
                        store_block(y, static_cast<uint8_t *>(p.a.out), (at + 32 * k) * 4, mine_ok);
                    } else {
                        if (mine_ok)
#pragma unroll
                            for (int x = 0; x < 32; x++) out[x] = y[x];
                        __syncwarp();   // whole warps load from tensor memory
                    }
                }
            }
            if (p.qs) {
                const int64_t block0 = row * p.row_blocks + head * NB + k0;
#pragma unroll 1
                for (int k = 0; k < NB / 2; k++) {
                    float y[32];
                    block_of(k0 + k, y);
                    float m = fabsf(y[0]);   // (a NaN row is NaN throughout: its scales are)
#pragma unroll
                    for (int x = 1; x < 32; x++) m = fmaxf(m, fabsf(y[x]));
                    const float d = m / 127.0f, rcp = 1.0f / d;
                    // rint(y / d): the product with 1 / d is within 127 * 2^-22 of the quotient, so divisions only where one
                    // of the block is next to a tie
                    bool tie = m < 0x1p-100f;
                    uint32_t w[8] = {};
#pragma unroll
                    for (int x = 0; x < 32; x++) {
                        const float z = y[x] * rcp, code = rintf(z);
                        tie |= fabsf(fabsf(z - code) - 0.5f) < 1e-4f;
                        w[x / 4] |= (uint32_t)((int)code & 255) << (8 * (x % 4));
                    }
                    if (tie) {
#pragma unroll
                        for (int x = 0; x < 32; x += 4) {
                            w[x / 4] = 0;
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                if (m != 0.0f) w[x / 4] |= (uint32_t)((int)rintf(y[x + e] / d) & 255) << (8 * e);
                        }
                    }
                    *reinterpret_cast<uint4 *>(staged<CH>(rows, lane, 2 * k)) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4 *>(staged<CH>(rows, lane, 2 * k + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
                    if (mine_ok) p.d[block0 + k] = __half_as_ushort(__float2half_rn(d));
                    __syncwarp();   // whole warps load from tensor memory
                }
                store_rows<CH, CH / 2>(rows, reinterpret_cast<uint8_t *>(p.qs), block0 * QB, mine_ok);
            }
            if (p.qs && there && ok && hf && head == p.a.n_heads - 1)   // the blocks behind the heads
                for (int64_t block = row * p.row_blocks + p.a.n_heads * NB; block < (row + 1) * p.row_blocks; block++) {
                    reinterpret_cast<uint4 *>(p.qs + block * QB)[0] = make_uint4(0, 0, 0, 0);
                    reinterpret_cast<uint4 *>(p.qs + block * QB)[1] = make_uint4(0, 0, 0, 0);
                    p.d[block] = 0;
                }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == MMA_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Tiles whose keys were shared out: one warp a row adds the shares in their order.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ PrefillArgs p) {
    constexpr int NB = D / 32, CTA_ROWS = Shape<D>::TILES * ROWS;
    pdl_trigger();
    pdl_wait();
    const int2 w = find_tile(p, blockIdx.x / p.c.Hkv, CTA_ROWS);
    if (w.x < 0) return;
    const Span1 sq = span_of(p, w.x);
    const int h = blockIdx.x % p.c.Hkv, lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int rho = w.y * CTA_ROWS + r;
    if (rho >= sq.n * p.G) return;
    const int token = rho / p.G, head = h * p.G + rho % p.G;
    const float sink = p.a.sinks ? ld_prev(p.a.sinks + head) * LOG2E : -INFINITY;
    const int64_t at = (int64_t)blockIdx.x * p.parts * CTA_ROWS + r;
    float top = sink, sum = 0.0f, o[NB];
#pragma unroll
    for (int k = 0; k < NB; k++) o[k] = 0.0f;
    for (int i0 = 0; i0 < p.parts; i0 += 32) {   // a lane a share
        const bool mine = i0 + lane < p.parts;
        const float2 *ml = p.part_ml + at + (int64_t)(i0 + lane) * CTA_ROWS;
        const float m = mine ? ld_prev(&ml->x) : -INFINITY, l = mine ? ld_prev(&ml->y) : 0.0f;
        float now = m;
#pragma unroll
        for (int x = 16; x; x >>= 1) now = fmaxf(now, __shfl_xor_sync(FULL, now, x));
        now = fmaxf(now, top);
        if (now == -INFINITY) {   // no keys so far: sums of 0, or NaN by the query
            if (__any_sync(FULL, l != l)) sum = NAN;
            continue;
        }
        const float old = top == -INFINITY ? 0.0f : ex2(top - now), f = m == -INFINITY ? 0.0f : ex2(m - now);
        top = now;
        float add = l * f;
#pragma unroll
        for (int x = 16; x; x >>= 1) add += __shfl_xor_sync(FULL, add, x);
        sum = fmaf(sum, old, add);
#pragma unroll
        for (int k = 0; k < NB; k++) o[k] *= old;
        const int some = min(32, p.parts - i0);
#pragma unroll 4
        for (int i = 0; i < some; i++) {
            const float g = __shfl_sync(FULL, f, i);
            const float *from = p.part_o + (at + (int64_t)(i0 + i) * CTA_ROWS) * D + lane;
#pragma unroll
            for (int k = 0; k < NB; k++) o[k] = fmaf(g > 0.0f ? ld_prev(from + 32 * k) : 0.0f, g, o[k]);   // (a share without keys has no outputs)
        }
    }
    if (sink != -INFINITY) sum += ex2(sink - top);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t row = sq.first + token;
#pragma unroll
    for (int k = 0; k < NB; k++) {
        const float y = o[k] * inv;
        const int64_t to = row * p.a.out_stride + (int64_t)head * D + 32 * k + lane;
        if (p.a.out && p.a.out_elem == QK_ELEM_F32) static_cast<float *>(p.a.out)[to] = y;
        if (p.a.out && p.a.out_elem == QK_ELEM_BF16) static_cast<__nv_bfloat16 *>(p.a.out)[to] = __float2bfloat16_rn(y);
        if (!p.qs) continue;
        float m = fabsf(y);
#pragma unroll
        for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, x));
        const float d = m / 127.0f;
        const int64_t block = row * p.row_blocks + head * NB + k;
        p.qs[block * QB + lane] = (int8_t)(m != 0.0f ? __float2int_rn(y / d) : 0);
        if (lane == 0) p.d[block] = __half_as_ushort(__float2half_rn(d));
    }
    if (p.qs && head == p.a.n_heads - 1)   // the blocks behind the heads
        for (int64_t block = row * p.row_blocks + p.a.n_heads * NB; block < (row + 1) * p.row_blocks; block++) {
            p.qs[block * QB + lane] = 0;
            if (lane == 0) p.d[block] = 0;
        }
}

// Shares of keys are for calls with fewer tiles than the device has room for; PART_CTAS bounds their number and so the
// workspace, and no call whose sequences are all shorter than PART_KEYS has any.
constexpr int PART_CTAS = 640, PART_KEYS = 2048;

struct Staged {
    int64_t lpad, k, v, there, part_o, part_ml, bytes;
};
Staged staged_of(int Hkv, int D, int64_t B, int64_t max_kv) {
    Staged l;
    l.lpad = ceil_div(max_kv, PAD) * PAD;
    l.k = 0;
    l.v = l.k + B * Hkv * l.lpad * D * 2;
    l.there = l.v + B * Hkv * l.lpad * D * 2;
    l.part_o = l.there + ceil_div(B * l.lpad / GROUP, 128) * 128;
    const int64_t rows = max_kv < PART_KEYS ? 0 : (int64_t)PART_CTAS * ROWS * (D == 256 ? 1 : 2);
    l.part_ml = l.part_o + rows * D * 4;
    l.bytes = l.part_ml + rows * 8;
    return l;
}

template <int D>
qk_status launch_tc(PrefillArgs &p, const Staged &l, cudaStream_t s) {
    using Z = Shape<D>;
    static bool ready[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fail(QK_ERR_CUDA, "attn_prefill: no device");
    if (!ready[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(attn_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
        if (e != cudaSuccess) return fail(QK_ERR_CUDA, "attn_prefill: %s", cudaGetErrorString(e));
        ready[dev] = true;
    }
    const auto encode = tensor_map_encoder();
    if (!encode) return fail(QK_ERR_CUDA, "attn_prefill: cuTensorMapEncodeTiled is not available");
    const auto map = [&](CUtensorMap *m, void *base, int64_t cols, int64_t rows, int box_rows) {
        const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, pitch[1] = {(cuuint64_t)cols * 2};
        const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
        return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, dims, pitch, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    const int64_t segs = (int64_t)p.B * p.c.Hkv;
    if (map(&p.kmap, p.k, D, segs * l.lpad, Z::BN) != CUDA_SUCCESS || map(&p.vmap, p.v, l.lpad, segs * D, D) != CUDA_SUCCESS)
        return fail(QK_ERR_CUDA, "attn_prefill: tensor map encoding failed");
    const qk_status st = launch_pdl("attn_stage", attn_stage_kernel<D>, dim3((unsigned)(l.lpad / 64), p.c.Hkv, p.B), dim3(128),
                                    0, s, p);
    if (st != QK_OK) return st;
    // tiles of any split of the rows into B sequences
    const int64_t tiles = (ceil_div((int64_t)p.rows * p.G, Z::TILES * ROWS) + std::min(p.B, p.rows) - 1) * p.c.Hkv;
    // Shares of keys: so many that rounds of CTAs times (steps of a share + what a CTA spends around them, about 8 steps)
    // is least, for keys as many as max_kv; a share is 4 steps at least. Whole calls, us, unshared / shared: 64 rows of 32
    // heads over 8 behind 60000 keys 714 / 125, 300 behind 4000 66 / 49, 1024 of 28 over 4 behind 32000 392 / 343.
    p.parts = 1;
    if (p.max_kv >= PART_KEYS) {
        const int64_t steps = ceil_div(p.max_kv, Z::BN), sms = sm_count();
        int64_t best = INT64_MAX;
        for (int n = 1; n == 1 || (n * tiles <= PART_CTAS && n * 4 <= steps); n++) {
            const int64_t cost = ceil_div(n * tiles, sms) * (ceil_div(steps, n) + 8 + (n > 1 ? 4 : 0));
            if (cost < best) best = cost, p.parts = n;
        }
    }
    const qk_status ran = launch_pdl("attn_prefill", attn_prefill_kernel<D>, dim3((unsigned)(tiles * p.parts)), dim3(Z::THREADS),
                                     (size_t)Z::SMEM, s, p);
    if (ran != QK_OK || p.parts == 1) return ran;
    return launch_pdl("attn_join", attn_join_kernel<D>, dim3((unsigned)tiles, Z::TILES * ROWS / 8), dim3(256), 0, s, p);
}

}  // namespace

int64_t attn_prefill_workspace_bytes(int Hkv, int D, int64_t B, int64_t max_kv) { return staged_of(Hkv, D, B, max_kv).bytes; }

qk_status launch_attn_prefill(const KvCache &c, const qk_attn &a, int B, int rows, const int32_t *q_offsets, int max_kv,
                              int8_t *qs, uint16_t *d, int64_t row_blocks, const int32_t *live, void *ws, cudaStream_t s) {
    const Staged l = staged_of(c.Hkv, c.D, B, max_kv);
    uint8_t *w = static_cast<uint8_t *>(ws);
    PrefillArgs p = {};
    p.c = c;
    p.a = a;
    p.B = B;
    p.rows = rows;
    p.G = a.n_heads / c.Hkv;
    p.max_kv = max_kv;
    p.lpad = (int)l.lpad;
    p.offsets = q_offsets;
    p.live = live;
    p.k = reinterpret_cast<__half *>(w + l.k);
    p.v = reinterpret_cast<__half *>(w + l.v);
    p.there = w + l.there;
    p.part_o = reinterpret_cast<float *>(w + l.part_o);
    p.part_ml = reinterpret_cast<float2 *>(w + l.part_ml);
    p.qs = qs;
    p.d = d;
    p.row_blocks = row_blocks;
    p.q_wide = row_wide(a.q, a.q_stride, a.q_elem);
    p.out16 = a.out && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_stride % 8 == 0;
    p.out_wide = a.out && row_wide(a.out, a.out_stride, a.out_elem);
    return c.D == 64 ? launch_tc<64>(p, l, s) : c.D == 128 ? launch_tc<128>(p, l, s) : launch_tc<256>(p, l, s);
}

qk_status read_attn_prefill_faults(uint32_t *faults) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tc_faults, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_tc_faults, &zero, sizeof zero);
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "qk_device_faults: %s", cudaGetErrorString(e));
    *faults = v;
    return QK_OK;
}

}  // namespace qk

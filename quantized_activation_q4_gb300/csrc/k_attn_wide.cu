// The decode attention of many query columns (heads of a group times new tokens: drafted tokens, wide groups): the pass of
// k_attn_decode.cu with one conversion of the codes for all of a CTA's columns.
//
// A CTA takes up to 32 columns. Of a tile of 64 tokens its four warps take 16 tokens each for the scores of all columns,
// leave the weights (binary16, as operands) in shared memory, and then take a quarter of the values' columns each for the
// weights of all tokens. So no code is converted twice, and a warp holds a quarter of the output: at D = 128 128 registers,
// four CTAs an SM. The warps keep one reference maximum a column between them. It moves only when a score is 2^8 above it,
// which they learn from each other by the barrier that the exchange needs anyway. Codes are converted exactly for both
// products (the bias of the scores as an initial accumulator would need more registers than there are).
//
// A group of 16 tokens of a head of 128 costs 874 warp instructions for 32 columns (the scales' products, exponentials and
// moves of 32 columns more than the conversion), issued half of the time (50%); most stalls are the fixed latency of dependent
// instructions (1.9 warps an issue), then copies (1.0) and shared memory (0.8). 16 sequences of 1500 to 9000 tokens with 8 new
// tokens each, 32 heads over 8: 67.2 us with the join; two CTAs of 16 columns in k_attn_decode.cu's kernel 66.0 (the rule at
// layout_of has both sides over more shapes). The conversions and products in one asm block, as there, spilled registers and
// took a microsecond more.

#include <algorithm>

#include "qk_decode.cuh"

namespace qk {
namespace {

constexpr int WARPS = 4;
constexpr int TILE = WIDE_TILE;
static_assert(TILE == WARPS * GROUP, "a group a warp");

template <int D, int NT>
struct Wide {
    static constexpr int NB = D / 32, W = NB < 4 ? NB : 4;
    static constexpr int MT = D / 16 / WARPS;              // column tiles (16) of the values a warp has
    static constexpr int S = D == 256 ? 2 : D == 128 ? 3 : 4;
    static constexpr int GB = group_bytes(D), STAGE = WARPS * GB;
    static constexpr int OFF_Q = S * STAGE;                // the queries' B operands: [block][column tile][lane] 16 bytes
    static constexpr int OFF_P = OFF_Q + NB * NT * 512;    // the weights': two tiles' [group][column tile][lane] 8 bytes
    static constexpr int SMEM = OFF_P + 2 * WARPS * NT * 256;
    static constexpr int PER_SM = D == 256 ? 2 : 4;
};

__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// Nibbles of bytes 0 and 2 of a word (low, high) less the bias of the exponents, exactly the codes less 8.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {
    const uint32_t v = (w & 0x000F000Fu) | 0x64006400u;
    const __half2 r = __hsub2(half2_bits(v), half2_bits(0x64086408u));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {
    const uint32_t v = (w & 0x00F000F0u) | 0x54005400u;
    const __half2 r = __hsub2(half2_bits(v), half2_bits(0x54805480u));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(WARPS * 32, Wide<D, NT>::PER_SM)
attn_wide_kernel(const __grid_constant__ DecodeArgs p, bool wide) {
    using Z = Wide<D, NT>;
    constexpr int NB = Z::NB, S = Z::S, GB = Z::GB, MT = Z::MT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan[WARPS];
    __shared__ int64_t found[2];
    __shared__ float column_scale[8 * NT];
    __shared__ float meet[WARPS][8 * NT];   // a column's largest score, or its sum, of each warp
    __shared__ int exponents[WARPS];        // of the largest scale of the values
    __shared__ __align__(4) uint8_t use[S][WARPS];
    __shared__ __align__(8) uint64_t bars[S];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int share = blockIdx.x / p.groups, cg = blockIdx.x % p.groups, shares = gridDim.x / p.groups;
    const int column0 = cg * 8 * NT;
    const uint32_t ring = smem_u32(smem), bar0 = smem_u32(&bars[0]), q_at = ring + Z::OFF_Q, p_at = ring + Z::OFF_P;
    if (threadIdx.x < S) mbar_init(bar0 + 8 * threadIdx.x, WARPS);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    // (no early start of the next kernel: see k_attn_decode.cu)
    pdl_wait();
    const int live = live_rows(p.live, p.B);
    Walk now;
    int64_t left = share_of<WARPS, TILE>(p, live, share, shares, scan, found, now);
    if (left <= 0) return;

    // what is on its way: one lane of every warp copies its group
    Walk ahead = now;
    int64_t to_issue = left;
    int page = -1, in_page = 0, table_at = 0, token = 0;   // of the next tile to issue
    bool ok = true;
    const auto place = [&]() {
        token = ahead.s.base + ahead.tile * TILE + warp * GROUP;
        table_at = token / p.c.page_tokens;
        in_page = token - table_at * p.c.page_tokens;
    };
    const auto look_up = [&]() {
        page = -1;
        if (lane == 0 && token < ahead.s.len)
            page = ld_prev(p.a.page_table + ahead.b * p.a.table_stride + table_at);
    };
    const auto issue = [&](int stage) {
        if (to_issue <= 0 || !ok) return;
        if (lane == 0) {
            const bool good = page >= 0 && page < p.c.n_pages;
            use[stage][warp] = good;
            if (good) {
                mbar_expect_tx(bar0 + 8 * stage, GB);
                bulk_g2s(ring + stage * Z::STAGE + warp * GB, group_at(p.c, page, ahead.h, in_page), GB, bar0 + 8 * stage);
            } else {
                mbar_arrive(bar0 + 8 * stage);
            }
        }
        if (--to_issue <= 0) return;
        next_tile<TILE>(ahead, p, live);
        if (ahead.tile == 0) {
            place();
        } else {   // a tile further on
            token += TILE;
            table_at += p.tile_pages;
            in_page += p.tile_rest;
            if (in_page >= p.c.page_tokens) {
                in_page -= p.c.page_tokens;
                table_at++;
            }
        }
        look_up();
    };
    place();
    look_up();
#pragma unroll
    for (int s = 0; s < S; s++) issue(s);

    float o[MT][NT][4], scale[NT][2], ref[NT][2], sum[NT][2], off[NT][2];
    int top_e = SMALLEST;   // exponent of the largest value scale so far
    bool fresh = true;    // a segment begins
    int stage = 0, buffer = 0, late = 0;
    int left_behind = -1;   // the stage of the tile before
    uint32_t parity = 0, late_parity = 0;
    for (;; left--) {
        if (fresh) {
            __syncthreads();   // (the queries of the segment before are no longer read)
            // warp w's column tiles: queries by a power of two less, as operands
            for (int n = warp; n < NT; n += WARPS) {
                const int col = column0 + 8 * n + g;
                const bool there = col < p.T * p.G;
                const int i = there ? col / p.G : 0, head = now.h * p.G + (there ? col % p.G : 0);
                const int64_t at = ((int64_t)now.b * p.T + i) * p.a.q_stride + (int64_t)head * D + 4 * t;
                const auto part = [&](int k, int e) {
                    const int64_t x = at + 32 * k + 16 * e;
                    float4 v = p.a.q_elem == QK_ELEM_F32 ? load_row4(static_cast<const float *>(p.a.q) + x, wide)
                                                         : load_row4(static_cast<const __nv_bfloat16 *>(p.a.q) + x, wide);
                    return there ? v : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                };
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < NB; k++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const float4 v = part(k, e);
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
                    }
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
                top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
                // 2^e is above the largest magnitude (above a quarter of it from 2^126 on); it and its inverse are normal numbers
                const int e2 = min(max((int)(__float_as_uint(top) >> 23) - 126, -126), 126);
                const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
                if (t == 0) column_scale[8 * n + g] = p.a.scale * __uint_as_float((uint32_t)(127 + e2) << 23) * LOG2E;
#pragma unroll
                for (int k = 0; k < NB; k++) {
                    const float4 x = part(k, 0), y = part(k, 1);
                    sts128(q_at + ((k * NT + n) * 32 + lane) * 16, pack2(x.x * down, x.z * down), pack2(x.y * down, x.w * down),
                           pack2(y.x * down, y.z * down), pack2(y.y * down, y.w * down));
                }
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    scale[n][e] = column_scale[8 * n + 2 * t + e];
                    ref[n][e] = -INFINITY;
                    off[n][e] = 0.0f;
                    sum[n][e] = 0.0f;
                }
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++) o[m][n][e] = 0.0f;
            top_e = SMALLEST;
            fresh = false;
        }
        if (ok) {
            ok = __all_sync(FULL, mbar_wait(bar0 + 8 * stage, parity));
            if (!ok) late = stage, late_parity = parity;
        }
        const uint32_t buf = ring + stage * Z::STAGE, mine = buf + warp * GB;
        const int token0 = now.s.base + now.tile * TILE;
        const int end0 = now.s.len - p.T + 1;   // keys that the first of the new tokens sees
        const int begin0 = p.a.window > 0 ? end0 - p.a.window : 0;   // no token sees a key below
        const uint32_t used = ok ? *reinterpret_cast<const uint32_t *>(&use[stage][0]) : 0;   // a byte a group
        const bool whole = used == 0x01010101u && token0 + TILE <= end0 && (p.a.window == 0 || token0 >= now.s.len - p.a.window);

        // the scores of the warp's group, times log2 e
        float s[NT][4];
        {
            uint64_t s2[NT][2];   // two columns each
            uint32_t dk[2][NB / 2];
            lds_words<NB / 2>(mine + 8 * D + 2 * NB * g, dk[0]);
            lds_words<NB / 2>(mine + 8 * D + 2 * NB * (g + 8), dk[1]);
#pragma unroll
            for (int bq = 0; bq < NB / Z::W; bq++) {
                uint32_t w0[Z::W], w1[Z::W];
                lds_words<Z::W>(mine + ((bq * GROUP + g) * 4 + t) * 4 * Z::W, w0);
                lds_words<Z::W>(mine + ((bq * GROUP + g + 8) * 4 + t) * 4 * Z::W, w1);
#pragma unroll
                for (int k = 0; k < Z::W; k++) {
                    const int b = bq * Z::W + k;
                    const float2 p0 = __half22float2(half2_bits(dk[0][b / 2])), p1 = __half22float2(half2_bits(dk[1][b / 2]));
                    const float d0 = b & 1 ? p0.y : p0.x, d1 = b & 1 ? p1.y : p1.x;
                    const uint64_t dd0 = two(d0, d0), dd1 = two(d1, d1);
                    const uint32_t lo[4] = {low_codes(w0[k]), low_codes(w1[k]), low_codes(w0[k] >> 8), low_codes(w1[k] >> 8)};
                    const uint32_t hi[4] = {high_codes(w0[k]), high_codes(w1[k]), high_codes(w0[k] >> 8), high_codes(w1[k] >> 8)};
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        const uint4 q = lds128(q_at + ((b * NT + n) * 32 + lane) * 16);
                        float a[4];
                        mma16_first(a, lo, q.x, q.y);
                        mma16(a, hi, q.z, q.w);
                        const uint64_t a0 = two(a[0], a[1]), a1 = two(a[2], a[3]);
                        s2[n][0] = fma2(dd0, a0, b == 0 ? 0 : s2[n][0]);
                        s2[n][1] = fma2(dd1, a1, b == 0 ? 0 : s2[n][1]);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int f = 0; f < 2; f++) {
                    const float2 x = apart(s2[n][f]);
                    s[n][2 * f] = x.x * scale[n][0];
                    s[n][2 * f + 1] = x.y * scale[n][1];
                }
        }
        bool move = false;
        if (!whole) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int end = min(end0 + (column0 + 8 * n + 2 * t + e) / p.G, now.s.len);
                    const int begin = p.a.window > 0 ? end - p.a.window : 0;
#pragma unroll
                    for (int f = 0; f < 2; f++) {
                        const int j = token0 + warp * GROUP + 8 * f + g;
                        if (!(used >> (8 * warp) & 1) || j >= end || j < begin) s[n][2 * f + e] = -INFINITY;
                    }
                }
        }
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) move |= fmaxf(s[n][e], s[n][2 + e]) - ref[n][e] > HEADROOM;   // (no: both minus infinity)
        const uint32_t scales = mine + 17 * D;   // the values', of the warp's group
        if (!whole) hide_scales<NB, 1>(scales, begin0 - token0 - warp * GROUP, now.s.len - token0 - warp * GROUP, used >> (8 * warp));
        const bool large = large_scales<NB, 1>(scales) || !usual(top_e);   // a scale of 2 or more, or unusual ones so far
        // All warps meet: what the tile before left in shared memory has been read, and whether something moves.
        if (__syncthreads_or(move || large)) {
            float top[NT][2];
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float x = fmaxf(s[n][e], s[n][2 + e]);
                    x = fmaxf(x, __shfl_xor_sync(FULL, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(FULL, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(FULL, x, 16));
                    if (g == 0) meet[warp][8 * n + 2 * t + e] = x;
                }
            const int mine_e = largest_exponent<NB, 1>(scales, top_e);
            if (lane == 0) exponents[warp] = mine_e;
            __syncthreads();
            int e_new = top_e;
#pragma unroll
            for (int w = 0; w < WARPS; w++) {
                e_new = max(e_new, exponents[w]);
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const float x = meet[w][8 * n + 2 * t + e];
                        top[n][e] = w == 0 ? x : fmaxf(top[n][e], x);
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float r = fmaxf(ref[n][e], top[n][e]);
                    // (rounded up, never below: weights stay under 2^14)
                    const float unit = r == -INFINITY ? 0.0f : __fadd_ru(r, (float)lift_of(e_new) - LIFT);
                    const float down = ref[n][e] == -INFINITY ? 0.0f : ex2(off[n][e] - unit);
                    ref[n][e] = r;
                    off[n][e] = unit;
                    sum[n][e] *= down;
#pragma unroll
                    for (int x = 0; x < MT; x++) {
                        o[x][n][e] *= down;
                        o[x][n][2 + e] *= down;
                    }
                }
            if (boost_of(e_new) != boost_of(top_e)) {
                const float change = power_of_two(boost_of(e_new) - boost_of(top_e));
#pragma unroll
                for (int x = 0; x < MT; x++)
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int e = 0; e < 4; e++) o[x][n][e] *= change;
            }
            top_e = e_new;
            if (!usual(top_e)) boost_scales<NB, 1>(scales, boost_of(top_e));   // (read by others after the next barrier)
        }
        // the tile before has been read by all: its stage is filled again
        if (left_behind >= 0) issue(left_behind);
        const uint32_t weights = p_at + buffer * WARPS * NT * 256;
#pragma unroll
        for (int n = 0; n < NT; n++) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                w[e] = ex2(s[n][e] - off[n][e & 1]);
                sum[n][e & 1] += w[e];
            }
            sts64(weights + ((warp * NT + n) * 32 + lane) * 8, transpose8(pack2(w[0], w[1])), transpose8(pack2(w[2], w[3])));
        }
        __syncthreads();
        // the outputs of the warp's column tiles
#pragma unroll
        for (int r = 0; r < WARPS; r++) {
            uint2 pt[NT];
#pragma unroll
            for (int n = 0; n < NT; n++) pt[n] = lds64(weights + ((r * NT + n) * 32 + lane) * 8);
            uint32_t x[MT];   // the words of its column tiles lie side by side
            lds_words<MT>(buf + r * GB + 9 * D + ((warp * MT / 4 * 8 + g) * 4 + t) * 16 + warp * MT % 4 * 4, x);
#pragma unroll
            for (int b = 0; b < (MT + 1) / 2; b++) {
                const uint2 d = lds64(buf + r * GB + 17 * D + (t * NB + warp * MT / 2 + b) * 8);   // tokens 2t, 2t + 1; 2t + 8, 2t + 9
                uint32_t pb[NT][2];
#pragma unroll
                for (int n = 0; n < NT; n++) pb[n][0] = mul2(pt[n].x, d.x), pb[n][1] = mul2(pt[n].y, d.y);
#pragma unroll
                for (int m = 2 * b; m < 2 * b + 2 && m < MT; m++) {
                    const uint32_t a[4] = {low_codes(x[m]), high_codes(x[m]), low_codes(x[m] >> 8), high_codes(x[m] >> 8)};
#pragma unroll
                    for (int n = 0; n < NT; n++) mma16(o[m][n], a, pb[n][0], pb[n][1]);
                }
            }
        }
        buffer ^= 1;
        if (left == 1 || now.tile + 1 == now.s.tiles) {
            // the segment ends here: its sums come together, its outputs are the warps' own
            const int64_t slot = ((int64_t)now.b * p.c.Hkv + now.h + share) * p.groups + cg;
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float l = sum[n][e];
                    l += __shfl_xor_sync(FULL, l, 4);
                    l += __shfl_xor_sync(FULL, l, 8);
                    l += __shfl_xor_sync(FULL, l, 16);
                    if (g == 0) meet[warp][8 * n + 2 * t + e] = l;
                }
            __syncthreads();
            if (warp == 0 && g == 0) {
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int col = 8 * n + 2 * t + e;
                        p.ml[slot * NT * 8 + col] =
                            make_float2(ref[n][e] == -INFINITY ? -INFINITY : off[n][e],
                                        (meet[0][col] + meet[1][col]) + (meet[2][col] + meet[3][col]));
                    }
            }
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        p.acc[(slot * NT * 8 + 8 * n + 2 * t + (e & 1)) * D + 16 * (warp * MT + m) + 8 * (e >> 1) + g] =
                            o[m][n][e] * power_of_two(-boost_of(top_e));
            fresh = true;
        }
        if (left == 1) break;
        next_tile<TILE>(now, p, live);
        left_behind = stage;
        if (++stage == S) {
            stage = 0;
            parity ^= 1;
        }
    }
    if (!ok)   // a wait ran out (nothing was issued since by this warp): no copy may land after the CTA has gone
        for (int k = late; k < late + S; k++)
            if (!mbar_wait(bar0 + 8 * (k % S), k < S ? late_parity : late_parity ^ 1)) break;
}

template <int D, int NT>
qk_status launch(const DecodeArgs &p, cudaStream_t s) {
    using Z = Wide<D, NT>;
    static bool ready[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fail(QK_ERR_CUDA, "attn_decode: no device");
    if (!ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_wide_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
        if (e != cudaSuccess) return fail(QK_ERR_CUDA, "attn_decode: %s", cudaGetErrorString(e));
        ready[dev] = true;
    }
    const int shares = std::max(1, std::min(Z::PER_SM * sm_count(), MAX_CTAS) / p.groups);
    return launch_pdl("attn_decode", attn_wide_kernel<D, NT>, dim3((unsigned)shares * p.groups), dim3(WARPS * 32), Z::SMEM, s, p,
                      row_wide(p.a.q, p.a.q_stride, p.a.q_elem));
}

}  // namespace

qk_status launch_attn_wide(const DecodeArgs &p, int NT, cudaStream_t s) {
    if (p.c.D == 64) return launch<64, 4>(p, s);
    if (p.c.D == 128) return launch<128, 4>(p, s);
    return NT == 2 ? launch<256, 2>(p, s) : launch<256, 4>(p, s);
}

qk_status read_attn_wide_faults(uint32_t *faults) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tc_faults, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_tc_faults, &zero, sizeof zero);
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "qk_device_faults: %s", cudaGetErrorString(e));
    *faults = v;
    return QK_OK;
}

}  // namespace qk

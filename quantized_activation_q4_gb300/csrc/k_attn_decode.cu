// Attention of a few new tokens of many sequences over the 4-bit cache (qk_attn_decode).
//
// attn_decode_kernel: one pass over the keys and values. The tiles of all sequences, in the order (sequence, head, token),
// are cut into equal shares, one for each resident CTA, so sequences of any lengths fill the device. A CTA's warps take a
// part of a tile each, with a running maximum, sum and output of their own; at the end of a segment (a share's part of one
// sequence and head) they meet and leave one partial result. attn_combine_kernel adds the partial results of a head in the
// order of its tokens, so outputs do not depend on the run, and writes rows and image.
//
// The tokens of a group are the rows (M) of the products, up to 8 NT query columns (query heads of the key/value head
// times new tokens) their columns (N), so a group of seven heads wastes an eighth and not half. With the scales outside
// of the products the operands are the codes themselves:
//   S[token][column] = sum over blocks b of d_k[token][b] * (sum over the block of (code - 8) * q)
//   O[x][column]    += sum over tokens of (code - 8) * (P[token][column] * d_v[token][block of x])
// A nibble becomes a half by one logic operation (1024 + code, or 64 + code in a high nibble). For S the bias leaves as the
// initial accumulator, -(1032 or 72) * sum q, once per segment; for O it is subtracted (the weights' sum would cancel
// catastrophically over long sequences). Queries are divided by a power of two to stay inside binary16, whatever their
// size. Weights are held as 2^6 at the reference and up to 2^14, those below 2^-20 of the reference to 2^-31 of it; what
// happens where the values' scales are not between 2^-3 and 2 is in qk_decode.cuh.
//
// A tile is 128 tokens, 64 for each of two warps (four groups: the barrier, the votes and the places of pages are paid for
// once; with 32 tokens a warp and tile 64 sequences of 8192 keys took 84 us for 71 when it was chosen). Six CTAs an SM by
// registers (168) and shared memory (two stages a warp).
//
// 2304 bytes of cache (16 tokens of a head of 128) cost 279 warp instructions, at full issue 9.4 TB/s. 64 sequences of 8192
// keys, 28 heads over 4 of 128: 67.5 us = 4.5 TB/s, 67% of the measured copy rate. Neither is full (issue 55% active): most
// stalls are the fixed latency of dependent instructions (1.1 warps an issue), copies and page numbers (0.75) and the math
// pipes (0.6).

#include <algorithm>

#include "qk_decode.cuh"

namespace qk {
namespace {

constexpr int WARPS = 2;
constexpr int GROUPS = 4;                   // of a warp's share of a tile
constexpr int WARP_TOKENS = GROUPS * GROUP;
constexpr int TILE = WARPS * WARP_TOKENS;   // tokens

// column tiles of 8 a CTA takes at most
__host__ __device__ constexpr int column_tiles(int D) { return D == 256 ? 1 : 2; }
__host__ __device__ constexpr int stages(int D) { return D == 64 ? 4 : 2; }
// CTAs of an SM, by registers and shared memory
__host__ __device__ constexpr int per_sm(int D, int NT) { return D == 256 ? 3 : NT == 2 ? (D == 64 ? 5 : 4) : 6; }

// ---------------------------------------------------------------- fragments
// Words of one block of two token rows (8 apart) times a column tile's queries: 16 tokens x 32 columns. The conversions and
// the two MMAs are one asm block, so that the halves land in the operand registers without moves.
template <int NT>
__device__ __forceinline__ void block_scores(float (&d)[NT][4], uint32_t x0, uint32_t x1, const uint32_t (&q)[NT][2][2],
                                             const float (&start)[NT][4]) {
    static_assert(NT == 1 || NT == 2, "column tiles");
    if constexpr (NT == 1) {
        asm("{\n .reg .b32 y0, y1, p0, p1, p2, p3, r0, r1, r2, r3;\n"
            " shr.u32 y0, %4, 8;\n shr.u32 y1, %5, 8;\n"
            " lop3.b32 p0, %4, 0x000F000F, 0x64006400, 0xEA;\n lop3.b32 p1, %5, 0x000F000F, 0x64006400, 0xEA;\n"
            " lop3.b32 p2, y0, 0x000F000F, 0x64006400, 0xEA;\n lop3.b32 p3, y1, 0x000F000F, 0x64006400, 0xEA;\n"
            " mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {p0,p1,p2,p3}, {%6,%7}, {%10,%11,%12,%13};\n"
            " lop3.b32 r0, %4, 0x00F000F0, 0x54005400, 0xEA;\n lop3.b32 r1, %5, 0x00F000F0, 0x54005400, 0xEA;\n"
            " lop3.b32 r2, y0, 0x00F000F0, 0x54005400, 0xEA;\n lop3.b32 r3, y1, 0x00F000F0, 0x54005400, 0xEA;\n"
            " mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {r0,r1,r2,r3}, {%8,%9}, {%0,%1,%2,%3};\n}\n"
            : "=&f"(d[0][0]), "=&f"(d[0][1]), "=&f"(d[0][2]), "=&f"(d[0][3])
            : "r"(x0), "r"(x1), "r"(q[0][0][0]), "r"(q[0][0][1]), "r"(q[0][1][0]), "r"(q[0][1][1]), "f"(start[0][0]),
              "f"(start[0][1]), "f"(start[0][2]), "f"(start[0][3]));
    } else {
        asm("{\n .reg .b32 y0, y1, p0, p1, p2, p3, r0, r1, r2, r3;\n"
            " shr.u32 y0, %8, 8;\n shr.u32 y1, %9, 8;\n"
            " lop3.b32 p0, %8, 0x000F000F, 0x64006400, 0xEA;\n lop3.b32 p1, %9, 0x000F000F, 0x64006400, 0xEA;\n"
            " lop3.b32 p2, y0, 0x000F000F, 0x64006400, 0xEA;\n lop3.b32 p3, y1, 0x000F000F, 0x64006400, 0xEA;\n"
            " mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {p0,p1,p2,p3}, {%10,%11}, {%18,%19,%20,%21};\n"
            " mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%4,%5,%6,%7}, {p0,p1,p2,p3}, {%14,%15}, {%22,%23,%24,%25};\n"
            " lop3.b32 r0, %8, 0x00F000F0, 0x54005400, 0xEA;\n lop3.b32 r1, %9, 0x00F000F0, 0x54005400, 0xEA;\n"
            " lop3.b32 r2, y0, 0x00F000F0, 0x54005400, 0xEA;\n lop3.b32 r3, y1, 0x00F000F0, 0x54005400, 0xEA;\n"
            " mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {r0,r1,r2,r3}, {%12,%13}, {%0,%1,%2,%3};\n"
            " mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%4,%5,%6,%7}, {r0,r1,r2,r3}, {%16,%17}, {%4,%5,%6,%7};\n}\n"
            : "=&f"(d[0][0]), "=&f"(d[0][1]), "=&f"(d[0][2]), "=&f"(d[0][3]), "=&f"(d[1][0]), "=&f"(d[1][1]), "=&f"(d[1][2]),
              "=&f"(d[1][3])
            : "r"(x0), "r"(x1), "r"(q[0][0][0]), "r"(q[0][0][1]), "r"(q[0][1][0]), "r"(q[0][1][1]), "r"(q[1][0][0]),
              "r"(q[1][0][1]), "r"(q[1][1][0]), "r"(q[1][1][1]), "f"(start[0][0]), "f"(start[0][1]), "f"(start[0][2]),
              "f"(start[0][3]), "f"(start[1][0]), "f"(start[1][1]), "f"(start[1][2]), "f"(start[1][3]));
    }
}
// A word of value codes (four tokens of columns u and u + 8 of a column tile of 16) times the weights: o += (code - 8) p
template <int NT>
__device__ __forceinline__ void word_outputs(float (&o)[NT][4], uint32_t x, const uint32_t (&p)[NT][2]) {
    if constexpr (NT == 1) {
        asm("{\n .reg .b32 y, p0, p1, p2, p3;\n shr.u32 y, %4, 8;\n"
            " lop3.b32 p0, %4, 0x000F000F, 0x64006400, 0xEA;\n lop3.b32 p1, %4, 0x00F000F0, 0x54005400, 0xEA;\n"
            " lop3.b32 p2, y, 0x000F000F, 0x64006400, 0xEA;\n lop3.b32 p3, y, 0x00F000F0, 0x54005400, 0xEA;\n"
            " sub.f16x2 p0, p0, %7;\n sub.f16x2 p1, p1, %8;\n sub.f16x2 p2, p2, %7;\n sub.f16x2 p3, p3, %8;\n"
            " mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {p0,p1,p2,p3}, {%5,%6}, {%0,%1,%2,%3};\n}\n"
            : "+f"(o[0][0]), "+f"(o[0][1]), "+f"(o[0][2]), "+f"(o[0][3])
            : "r"(x), "r"(p[0][0]), "r"(p[0][1]), "r"(0x64086408u), "r"(0x54805480u));
    } else {
        asm("{\n .reg .b32 y, p0, p1, p2, p3;\n shr.u32 y, %8, 8;\n"
            " lop3.b32 p0, %8, 0x000F000F, 0x64006400, 0xEA;\n lop3.b32 p1, %8, 0x00F000F0, 0x54005400, 0xEA;\n"
            " lop3.b32 p2, y, 0x000F000F, 0x64006400, 0xEA;\n lop3.b32 p3, y, 0x00F000F0, 0x54005400, 0xEA;\n"
            " sub.f16x2 p0, p0, %13;\n sub.f16x2 p1, p1, %14;\n sub.f16x2 p2, p2, %13;\n sub.f16x2 p3, p3, %14;\n"
            " mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {p0,p1,p2,p3}, {%9,%10}, {%0,%1,%2,%3};\n"
            " mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%4,%5,%6,%7}, {p0,p1,p2,p3}, {%11,%12}, {%4,%5,%6,%7};\n}\n"
            : "+f"(o[0][0]), "+f"(o[0][1]), "+f"(o[0][2]), "+f"(o[0][3]), "+f"(o[1][0]), "+f"(o[1][1]), "+f"(o[1][2]),
              "+f"(o[1][3])
            : "r"(x), "r"(p[0][0]), "r"(p[0][1]), "r"(p[1][0]), "r"(p[1][1]), "r"(0x64086408u), "r"(0x54805480u));
    }
}
// The queries of a segment's columns as B operands, and what the scores need besides.
template <int D, int NT>
struct Queries {
    static constexpr int NB = D / 32;
    uint32_t b[NB][NT][2][2];    // [block][column tile][low, high nibbles][register]
    float start[NB][NT][4];      // -(bias * sum of the block's queries), columns 2t and 2t + 1, twice
    float scale[NT][2];          // scale * log2 e * the queries' power of two
};
template <int D, int NT>
__device__ __forceinline__ void load_queries(Queries<D, NT> &q, const DecodeArgs &p, int b, int h, int column0, bool wide) {
    constexpr int NB = D / 32;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; n++) {
        const int col = column0 + 8 * n + g;
        const bool there = col < p.T * p.G;
        const int i = there ? col / p.G : 0, head = h * p.G + (there ? col % p.G : 0);
        const int64_t at = ((int64_t)b * p.T + i) * p.a.q_stride + (int64_t)head * D;
        float4 x[NB][2];
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < NB; k++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int64_t o = at + 32 * k + 16 * e + 4 * t;
                x[k][e] = p.a.q_elem == QK_ELEM_F32
                              ? load_row4(static_cast<const float *>(p.a.q) + o, wide)
                              : load_row4(static_cast<const __nv_bfloat16 *>(p.a.q) + o, wide);
                if (!there) x[k][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                top = fmaxf(top, fmaxf(fmaxf(fabsf(x[k][e].x), fabsf(x[k][e].y)), fmaxf(fabsf(x[k][e].z), fabsf(x[k][e].w))));
            }
        top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
        top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
        // 2^e is above the largest magnitude (above a quarter of it from 2^126 on); it and its inverse are normal numbers
        const int e2 = min(max((int)(__float_as_uint(top) >> 23) - 126, -126), 126);
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23), up = __uint_as_float((uint32_t)(127 + e2) << 23);
        const float c = p.a.scale * up * LOG2E;   // (0 where the queries are 0 and it underflows: so are the scores)
#pragma unroll
        for (int k = 0; k < NB; k++) {
            float bias = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const __half2 v0 = __floats2half2_rn(x[k][e].x * down, x[k][e].z * down);   // nibbles of bytes 0 and 2
                const __half2 v1 = __floats2half2_rn(x[k][e].y * down, x[k][e].w * down);   // 1 and 3
                q.b[k][n][e][0] = *reinterpret_cast<const uint32_t *>(&v0);
                q.b[k][n][e][1] = *reinterpret_cast<const uint32_t *>(&v1);
                const float2 f0 = __half22float2(v0), f1 = __half22float2(v1);
                bias = fmaf(e ? -72.0f : -1032.0f, (f0.x + f0.y) + (f1.x + f1.y), bias);
            }
            bias += __shfl_xor_sync(FULL, bias, 1);
            bias += __shfl_xor_sync(FULL, bias, 2);
            q.start[k][n][0] = q.start[k][n][2] = __shfl_sync(FULL, bias, 8 * t);
            q.start[k][n][1] = q.start[k][n][3] = __shfl_sync(FULL, bias, 8 * t + 4);
        }
        q.scale[n][0] = __shfl_sync(FULL, c, 8 * t);
        q.scale[n][1] = __shfl_sync(FULL, c, 8 * t + 4);
    }
}

// ---------------------------------------------------------------- the pass
template <int D, int NT>
__global__ void __launch_bounds__(WARPS * 32, per_sm(D, NT))
attn_decode_kernel(const __grid_constant__ DecodeArgs p, bool wide) {
    constexpr int NB = D / 32, S = stages(D), GB = group_bytes(D), MT = D / 16, W = NB < 4 ? NB : 4;
    constexpr int STAGE = GROUPS * GB, PITCH = D + 4;
    static_assert(8 * PITCH * 4 <= STAGE, "a warp's partial outputs fit its stage");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t scan[WARPS];
    __shared__ int64_t found[2];
    __shared__ float2 meet[WARPS][8];
    __shared__ __align__(4) uint8_t use[WARPS][S][GROUPS];
    __shared__ __align__(8) uint64_t bars[WARPS][S];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int share = blockIdx.x / p.groups, cg = blockIdx.x % p.groups, shares = gridDim.x / p.groups;
    const int column0 = cg * 8 * NT;
    const uint32_t ring = smem_u32(smem) + warp * S * STAGE, bar0 = smem_u32(&bars[warp][0]);
    if (lane < S) mbar_init(bar0 + 8 * lane, GROUPS);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // (No early start of the next kernel: the join's CTAs, waiting on SMs that are done, held up the passes of calls in a row;
    // 64 sequences of 8192 keys took 93 us a call for 71 then.)
    pdl_wait();
    const int live = live_rows(p.live, p.B);

    Walk now;
    int64_t left = share_of<WARPS, TILE>(p, live, share, shares, scan, found, now);
    if (left <= 0) return;

    // what is on its way: the first lanes copy a group each
    Walk ahead = now;
    int64_t to_issue = left;
    int page = -1, in_page = 0, table_at = 0, token = 0;   // of the next tile to issue
    bool ok = true;
    const auto place = [&]() {   // of the first tile in a segment
        token = ahead.s.base + ahead.tile * TILE + warp * WARP_TOKENS + lane * GROUP;
        table_at = token / p.c.page_tokens;
        in_page = token - table_at * p.c.page_tokens;
    };
    const auto look_up = [&]() {
        page = -1;
        if (lane < GROUPS && token < ahead.s.len)
            page = ld_prev(p.a.page_table + ahead.b * p.a.table_stride + table_at);
    };
    const auto issue = [&](int stage) {
        if (to_issue <= 0 || !ok) return;
        if (lane < GROUPS) {
            const bool good = page >= 0 && page < p.c.n_pages;
            use[warp][stage][lane] = good;
            if (good) {
                mbar_expect_tx(bar0 + 8 * stage, GB);
                bulk_g2s(ring + stage * STAGE + lane * GB, group_at(p.c, page, ahead.h, in_page), GB, bar0 + 8 * stage);
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
    __syncwarp();
    place();
    look_up();
#pragma unroll
    for (int s = 0; s < S; s++) issue(s);

    float o[MT][NT][4], ref[NT][2], sum[NT][2], off[NT][2];
    Queries<D, NT> q;
    int top_e = SMALLEST;   // exponent of the largest value scale so far
    bool fresh = true;    // a segment begins
    int stage = 0;
    uint32_t parity = 0, late_parity = 0;
    int late = 0;         // where a wait ran out
    for (;; left--) {
        if (fresh) {
            load_queries<D, NT>(q, p, now.b, now.h, column0, wide);
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
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
        const uint32_t buf = ring + stage * STAGE;
        const int token0 = now.s.base + now.tile * TILE + warp * WARP_TOKENS;
        const int end0 = now.s.len - p.T + 1;   // keys that the first of the new tokens sees
        const int begin0 = p.a.window > 0 ? end0 - p.a.window : 0;   // no token sees a key below
        // scores, times log2 e
        float s[GROUPS][NT][4];
        uint32_t used = 0;
        if (ok) used = *reinterpret_cast<const uint32_t *>(&use[warp][stage][0]);   // a byte a group
#pragma unroll
        for (int r = 0; r < GROUPS; r++) {
            const uint32_t grp = buf + r * GB;
            uint32_t dk[2][NB / 2];
            lds_words<NB / 2>(grp + 8 * D + 2 * NB * g, dk[0]);
            lds_words<NB / 2>(grp + 8 * D + 2 * NB * (g + 8), dk[1]);
#pragma unroll
            for (int bq = 0; bq < NB / W; bq++) {
                uint32_t w0[W], w1[W];
                lds_words<W>(grp + ((bq * GROUP + g) * 4 + t) * 4 * W, w0);
                lds_words<W>(grp + ((bq * GROUP + g + 8) * 4 + t) * 4 * W, w1);
#pragma unroll
                for (int k = 0; k < W; k++) {
                    const int b = bq * W + k;
                    const float2 p0 = __half22float2(half2_bits(dk[0][b / 2])), p1 = __half22float2(half2_bits(dk[1][b / 2]));
                    const float d0 = b & 1 ? p0.y : p0.x, d1 = b & 1 ? p1.y : p1.x;
                    float a[NT][4];
                    block_scores<NT>(a, w0[k], w1[k], q.b[b], q.start[b]);
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            s[r][n][e] = b == 0 ? (e < 2 ? d0 : d1) * a[n][e] : fmaf(e < 2 ? d0 : d1, a[n][e], s[r][n][e]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) s[r][n][e] *= q.scale[n][e & 1];
        }
        // some query does not see some key, or a group's page does not exist (what its stage holds is masked)
        const bool whole = used == 0x01010101u && token0 + WARP_TOKENS <= end0 &&
                           (p.a.window == 0 || token0 >= now.s.len - p.a.window);
        if (!whole) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int end = min(end0 + (column0 + 8 * n + 2 * t + e) / p.G, now.s.len);
                    const int begin = p.a.window > 0 ? end - p.a.window : 0;
#pragma unroll
                    for (int r = 0; r < GROUPS; r++)
#pragma unroll
                        for (int f = 0; f < 2; f++) {
                            const int j = token0 + r * GROUP + 8 * f + g;
                            if (!(used >> (8 * r) & 1) || j >= end || j < begin) s[r][n][2 * f + e] = -INFINITY;
                        }
                }
        }
        // the lane's maxima of its columns; the reference moves only far
        float top[NT][2];
        bool move = false;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float m = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
                for (int r = 1; r < GROUPS; r++) m = fmaxf(fmaxf(m, s[r][n][e]), s[r][n][2 + e]);
                top[n][e] = m;
                move |= m - ref[n][e] > HEADROOM;   // (no: both are minus infinity)
            }
        const uint32_t scales = buf + 17 * D;   // the values', of the first group
        if (!whole) hide_scales<NB, GROUPS>(scales, begin0 - token0, now.s.len - token0, used);
        const bool large = large_scales<NB, GROUPS>(scales) || !usual(top_e);   // a scale of 2 or more, or unusual ones so far
        int e_new = top_e;
        if (__any_sync(FULL, move || large)) {
            if (__any_sync(FULL, large)) {
                e_new = largest_exponent<NB, GROUPS>(scales, top_e);
                if (!usual(e_new)) boost_scales<NB, GROUPS>(scales, boost_of(e_new));
            }
        }
        if (__any_sync(FULL, move) || e_new != top_e) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float m = top[n][e];
                    m = fmaxf(m, __shfl_xor_sync(FULL, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(FULL, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(FULL, m, 16));
                    const float r = fmaxf(ref[n][e], m);
                    // (rounded up, never below: weights stay under 2^14)
                    const float unit = r == -INFINITY ? 0.0f : __fadd_ru(r, (float)lift_of(e_new) - LIFT);
                    const float down = ref[n][e] == -INFINITY ? 0.0f : ex2(off[n][e] - unit);
                    ref[n][e] = r;
                    off[n][e] = unit;
                    sum[n][e] *= down;
#pragma unroll
                    for (int m = 0; m < MT; m++) {
                        o[m][n][e] *= down;
                        o[m][n][2 + e] *= down;
                    }
                }
            if (boost_of(e_new) != boost_of(top_e)) {
                const float change = power_of_two(boost_of(e_new) - boost_of(top_e));
#pragma unroll
                for (int m = 0; m < MT; m++)
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int e = 0; e < 4; e++) o[m][n][e] *= change;
            }
            top_e = e_new;
        }
#pragma unroll
        for (int r = 0; r < GROUPS; r++) {
            const uint32_t grp = buf + r * GB;
            uint32_t dv[2 * NB];
            lds_words<2 * NB>(scales + r * GB + t * 8 * NB, dv);
            uint32_t pt[NT][2];   // weights of query g: tokens 2t, 2t + 1 and 2t + 8, 2t + 9
#pragma unroll
            for (int n = 0; n < NT; n++) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    w[e] = ex2(s[r][n][e] - off[n][e & 1]);
                    sum[n][e & 1] += w[e];
                }
                pt[n][0] = transpose8(pack2(w[0], w[1]));
                pt[n][1] = transpose8(pack2(w[2], w[3]));
            }
#pragma unroll
            for (int mq = 0; mq < MT / 4; mq++) {
                uint32_t w[4];
                lds_words<4>(grp + 9 * D + ((mq * 8 + g) * 4 + t) * 16, w);
#pragma unroll
                for (int bb = 0; bb < 2; bb++) {
                    const int b = 2 * mq + bb;
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        pb[n][0] = mul2(pt[n][0], dv[2 * b]);
                        pb[n][1] = mul2(pt[n][1], dv[2 * b + 1]);
                    }
#pragma unroll
                    for (int mm = 0; mm < 2; mm++) word_outputs<NT>(o[2 * b + mm], w[2 * bb + mm], pb);
                }
            }
        }
        __syncwarp();   // the stage is read
        if (left == 1 || now.tile + 1 == now.s.tiles) {
            // the segment ends here: one partial result of the warps, through the stages just read
            const int64_t slot = ((int64_t)now.b * p.c.Hkv + now.h + share) * p.groups + cg;
#pragma unroll
            for (int n = 0; n < NT; n++) {
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float l = sum[n][e];
                    l += __shfl_xor_sync(FULL, l, 4);
                    l += __shfl_xor_sync(FULL, l, 8);
                    l += __shfl_xor_sync(FULL, l, 16);
                    if (g == 0) meet[warp][2 * t + e] = make_float2(ref[n][e] == -INFINITY ? -INFINITY : off[n][e], l);
                }
                __syncthreads();
                float down[2];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float m = -INFINITY;
#pragma unroll
                    for (int w = 0; w < WARPS; w++) m = fmaxf(m, meet[w][2 * t + e].x);
                    down[e] = ref[n][e] == -INFINITY ? 0.0f : ex2(off[n][e] - m) * power_of_two(-boost_of(top_e));
                }
                float *mine = reinterpret_cast<float *>(smem + (warp * S + stage) * STAGE);
#pragma unroll
                for (int m = 0; m < MT; m++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        mine[(2 * t + (e & 1)) * PITCH + 16 * m + 8 * (e >> 1) + g] = o[m][n][e] * down[e & 1];
                __syncthreads();
                const float *all = reinterpret_cast<const float *>(smem + stage * STAGE);
                constexpr int STEP = S * STAGE / 4;   // floats from one warp's stage to the next one's
                float *out = p.acc + (slot * NT + n) * 8 * D;
                for (int i = threadIdx.x; i < 8 * D; i += WARPS * 32) {
                    const int at = i / D * PITCH + i % D;
                    float v = all[at];
#pragma unroll
                    for (int w = 1; w < WARPS; w++) v += all[at + w * STEP];
                    out[i] = v;
                }
                if (threadIdx.x < 8) {
                    float m = -INFINITY, l = 0.0f;
#pragma unroll
                    for (int w = 0; w < WARPS; w++) m = fmaxf(m, meet[w][threadIdx.x].x);
#pragma unroll
                    for (int w = 0; w < WARPS; w++) {
                        const float2 v = meet[w][threadIdx.x];
                        l += v.y * (v.x == -INFINITY ? 0.0f : ex2(v.x - m));   // (NaN stays)
                    }
                    p.ml[(slot * NT + n) * 8 + threadIdx.x] = make_float2(m, l);
                }
                __syncthreads();
            }
            fresh = true;
        }
        if (left == 1) break;
        next_tile<TILE>(now, p, live);
        // the stage was read and written by plain accesses; the next copy into it comes after them
        if (fresh) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        issue(stage);
        if (++stage == S) {
            stage = 0;
            parity ^= 1;
        }
    }
    if (!ok)   // a wait ran out (nothing was issued since): no copy may land after the CTA has gone
        for (int k = late; k < late + S; k++)
            if (!mbar_wait(bar0 + 8 * (k % S), k < S ? late_parity : late_parity ^ 1)) break;
}

// ---------------------------------------------------------------- joining
struct JoinArgs {
    DecodeArgs p;
    uint8_t *img;
    int64_t row_blocks;
    int NT, tile;
};
// A lane's column of block k of a head: its row and image.
template <int NB>
__device__ __forceinline__ void put_block(const JoinArgs &a, int row, int head, int k, float y) {
    const qk_attn &out = a.p.a;
    const int lane = threadIdx.x & 31;
    const int64_t to = row * out.out_stride + (int64_t)head * 32 * NB + 32 * k + lane;
    if (out.out && out.out_elem == QK_ELEM_F32) static_cast<float *>(out.out)[to] = y;
    if (out.out && out.out_elem == QK_ELEM_BF16) static_cast<__nv_bfloat16 *>(out.out)[to] = __float2bfloat16_rn(y);
    if (!a.img) return;
    float m = fabsf(y);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, x));
    const float d = m / 127.0f;
    const int code = m != 0.0f ? __float2int_rn(y / d) : 0;
    const int sum = __reduce_add_sync(FULL, code);
    uint8_t *block = a.img + (row * a.row_blocks + (int64_t)head * NB + k) * Q8_1_BYTES;
    block[4 + lane] = (uint8_t)code;
    if (lane == 0) *reinterpret_cast<__half2 *>(block) = __halves2half2(__float2half_rn(d), __float2half_rn(d * (float)sum));
}
// The blocks behind a row's heads, by the last head's threads.
template <int NB>
__device__ __forceinline__ void clear_behind(const JoinArgs &a, int row, int thread, int threads) {
    if (!a.img) return;
    uint32_t *rest = reinterpret_cast<uint32_t *>(a.img + (row * a.row_blocks + (int64_t)a.p.a.n_heads * NB) * Q8_1_BYTES);
    const int64_t words = (a.row_blocks - (int64_t)a.p.a.n_heads * NB) * (Q8_1_BYTES / 4);
    for (int64_t x = thread; x < words; x += threads) rest[x] = 0;
}

// One CTA per (row, query head): the statistics of all partial results first, then their outputs in order, four warps side
// by side with several loads under way; then rows and image.
constexpr int JOIN_WARPS = 4;
template <int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) attn_combine_kernel(const __grid_constant__ JoinArgs a) {
    constexpr int NB = D / 32;
    __shared__ float part[JOIN_WARPS][D];
    __shared__ float reduce[JOIN_WARPS];
    pdl_trigger();
    pdl_wait();
    const DecodeArgs &p = a.p;
    const int head = blockIdx.x, row = blockIdx.y;
    const int b = row / p.T, i = row % p.T, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (b >= p.B) return;
    const int h = head / p.G, col = i * p.G + head % p.G;
    // (loaded together: the live count, the length, the sink and the plan, which holds something for live sequences alone)
    const int live = live_rows(p.live, p.B);
    const Sequence s = a.tile == TILE ? sequence_of<TILE>(p, b) : sequence_of<WIDE_TILE>(p, b);
    const float sink = p.a.sinks ? ld_prev(p.a.sinks + head) * LOG2E : -INFINITY;
    const int64_t each = ld_prev(p.plan), tiles_before = ld_prev(p.plan + 1 + b);
    if (b >= live) return;
    const int64_t lo = tiles_before + (int64_t)h * s.tiles, c0 = s.tiles > 0 ? lo / each : 0;
    const int count = s.tiles > 0 ? (int)((lo + s.tiles - 1) / each - c0) + 1 : 0;
    const int n = col / 8, cg = n / a.NT;
    const int64_t step = (int64_t)p.groups * a.NT * 8;   // from one partial result to the next
    const int64_t at = (((int64_t)b * p.c.Hkv + h + c0) * p.groups + cg) * a.NT * 8 + n % a.NT * 8 + col % 8;
    const auto over_cta = [&](float v, bool largest) {
#pragma unroll
        for (int m = 16; m; m >>= 1) {
            const float w = __shfl_xor_sync(FULL, v, m);
            v = largest ? fmaxf(v, w) : v + w;
        }
        __syncthreads();
        if (lane == 0) reduce[warp] = v;
        __syncthreads();
        v = reduce[0];
#pragma unroll
        for (int w = 1; w < JOIN_WARPS; w++) v = largest ? fmaxf(v, reduce[w]) : v + reduce[w];
        return v;
    };
    float top = sink;
    for (int c = threadIdx.x; c < count; c += JOIN_WARPS * 32) top = fmaxf(top, ld_prev(&p.ml[at + c * step].x));
    top = over_cta(top, true);
    float total = 0.0f;
    const auto factor = [&](int c) {
        const float m = ld_prev(&p.ml[at + c * step].x);
        return m == -INFINITY ? 0.0f : ex2(m - top);
    };
    for (int c = threadIdx.x; c < count; c += JOIN_WARPS * 32) {
        const float f = factor(c);
        total = fmaf(ld_prev(&p.ml[at + c * step].y), f, total);
    }
    total = over_cta(total, false);
    if (sink != -INFINITY) total += ex2(sink - top);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;   // no key and no sink: 0
    float o[NB];
#pragma unroll
    for (int k = 0; k < NB; k++) o[k] = 0.0f;
#pragma unroll 4
    for (int c = warp; c < count; c += JOIN_WARPS) {
        const float f = factor(c);
#pragma unroll
        for (int k = 0; k < NB; k++) o[k] = fmaf(ld_prev(p.acc + (at + c * step) * D + 32 * k + lane), f, o[k]);
    }
#pragma unroll
    for (int k = 0; k < NB; k++) part[warp][32 * k + lane] = o[k];
    __syncthreads();
    for (int k = warp; k < NB; k += JOIN_WARPS) {
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; w++) y += part[w][32 * k + lane];
        put_block<NB>(a, row, head, k, y * inv);
    }
    if (head == p.a.n_heads - 1) clear_behind<NB>(a, row, threadIdx.x, JOIN_WARPS * 32);
}

// Many rows and heads, few partial results of each: a warp a head, 32 statistics at once.
template <int D>
__global__ void __launch_bounds__(128) attn_combine_warps_kernel(const __grid_constant__ JoinArgs a) {
    constexpr int NB = D / 32;
    pdl_trigger();
    pdl_wait();
    const DecodeArgs &p = a.p;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int row = (int)(unit / p.a.n_heads), head = (int)(unit - (int64_t)row * p.a.n_heads), lane = threadIdx.x & 31;
    const int b = row / p.T, i = row - b * p.T;
    if (b >= p.B) return;
    const int live = live_rows(p.live, p.B);
    const Sequence s = a.tile == TILE ? sequence_of<TILE>(p, b) : sequence_of<WIDE_TILE>(p, b);
    const float sink = p.a.sinks ? ld_prev(p.a.sinks + head) * LOG2E : -INFINITY;
    const int64_t each = ld_prev(p.plan), tiles_before = ld_prev(p.plan + 1 + b);
    if (b >= live) return;
    const int h = head / p.G, col = i * p.G + head - h * p.G;
    const int64_t lo = tiles_before + (int64_t)h * s.tiles, c0 = s.tiles > 0 ? lo / each : 0;
    const int count = s.tiles > 0 ? (int)((lo + s.tiles - 1) / each - c0) + 1 : 0;
    const int n = col / 8, cg = n / a.NT;
    const int64_t step = (int64_t)p.groups * a.NT * 8;   // from one partial result to the next
    const int64_t at = (((int64_t)b * p.c.Hkv + h + c0) * p.groups + cg) * a.NT * 8 + n % a.NT * 8 + col % 8;
    float top = sink, total = 0.0f, o[NB];
#pragma unroll
    for (int k = 0; k < NB; k++) o[k] = 0.0f;
    for (int first = 0; first < count; first += 32) {
        const bool mine = first + lane < count;
        const float2 *ml = p.ml + at + (int64_t)(first + lane) * step;
        const float m = mine ? ld_prev(&ml->x) : -INFINITY, l = mine ? ld_prev(&ml->y) : 0.0f;
        float now = m;
#pragma unroll
        for (int x = 16; x; x >>= 1) now = fmaxf(now, __shfl_xor_sync(FULL, now, x));
        now = fmaxf(now, top);
        if (now == -INFINITY) {   // no keys so far: sums of 0, or NaN by the query
            if (__any_sync(FULL, l != l)) total = NAN;
            continue;
        }
        const float old = top == -INFINITY ? 0.0f : ex2(top - now), f = m == -INFINITY ? 0.0f : ex2(m - now);
        top = now;
        float add = l * f;
#pragma unroll
        for (int x = 16; x; x >>= 1) add += __shfl_xor_sync(FULL, add, x);
        total = fmaf(total, old, add);
#pragma unroll
        for (int k = 0; k < NB; k++) o[k] *= old;
        const int some = min(32, count - first);
#pragma unroll 4
        for (int c = 0; c < some; c++) {
            const float g = __shfl_sync(FULL, f, c);
#pragma unroll
            for (int k = 0; k < NB; k++) o[k] = fmaf(ld_prev(p.acc + (at + (first + c) * step) * D + 32 * k + lane), g, o[k]);
        }
    }
    if (sink != -INFINITY) total += ex2(sink - top);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;   // no key and no sink: 0
#pragma unroll
    for (int k = 0; k < NB; k++) put_block<NB>(a, row, head, k, o[k] * inv);
    if (head == p.a.n_heads - 1) clear_behind<NB>(a, row, lane, 32);
}

struct Layout {
    int NT, groups, tile;   // tile: of the kernel that the call takes
    int64_t slots, acc, ml, plan, bytes;
};
Layout layout_of(int Hkv, int D, int n_heads, int64_t B, int T) {
    Layout l;
    const int tiles = (T * (n_heads / Hkv) + 7) / 8;   // of 8 columns
    // Up to 16 columns (8 at head_dim 256, for the registers of the output) take this file's kernel, more the wide one.
    // Both sides, us, this file's (CTAs of up to 16 columns, 8 at D = 256) / the wide one's (32; 16 at D = 256 if they do):
    //   32 sequences of 8192 keys: 16 columns, D = 128, 2 kv heads 45 / 61; 14, D = 128, 4: 65 / 97; 16, D = 64, 8: 70 / 115
    //   16 sequences of 8192 keys, D = 256: 8 columns, 4 kv heads 55 / 70; 16, 2: 51 / 48
    //   16 sequences of 1500 to 9000 keys: 17, 24, 32 columns of 8 kv heads, D = 64 49.5, 50.2, 50.5 / 47.9, 48.8, 49.3;
    //   D = 128 72.8, 73.7, 73.1 / 73.5, 74.9, 74.9; D = 256, 4 kv heads: 12 columns 62 / 55, 32: 102 / 70
    // At D = 128 it is close: 2 sequences of 2000 keys, 32 columns of 8 kv heads 16.0 / 17.1, 64 of 1000, 20 columns 78 / 65.
    const bool wide = tiles > column_tiles(D);
    l.NT = wide ? (tiles > 2 ? WIDE_COLUMNS : 2) : tiles;
    l.groups = (tiles + l.NT - 1) / l.NT;
    l.tile = wide ? WIDE_TILE : TILE;
    // segments and shares interleave, so (segment + share) names each part of a segment once
    l.slots = (B * Hkv + MAX_CTAS) * l.groups;
    l.acc = 0;
    l.ml = l.acc + l.slots * l.NT * 8 * D * 4;
    l.plan = l.ml + l.slots * l.NT * 8 * 8;
    l.bytes = l.plan + (1 + B) * 8;
    return l;
}

template <int D, int NT>
qk_status launch_pass(const DecodeArgs &p, cudaStream_t s) {
    constexpr int smem = WARPS * stages(D) * GROUPS * group_bytes(D);
    static bool ready[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fail(QK_ERR_CUDA, "attn_decode: no device");
    if (!ready[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(attn_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return fail(QK_ERR_CUDA, "attn_decode: %s", cudaGetErrorString(e));
        ready[dev] = true;
    }
    const int shares = std::max(1, std::min(per_sm(D, NT) * sm_count(), MAX_CTAS) / p.groups);
    const bool wide = row_wide(p.a.q, p.a.q_stride, p.a.q_elem);
    return launch_pdl("attn_decode", attn_decode_kernel<D, NT>, dim3((unsigned)shares * p.groups), dim3(WARPS * 32), smem, s,
                      p, wide);
}

}  // namespace

int64_t attn_decode_workspace_bytes(int Hkv, int D, int n_heads, int64_t B, int T) {
    return layout_of(Hkv, D, n_heads, B, T).bytes;
}

qk_status launch_attn_decode(const KvCache &c, const qk_attn &a, int B, int T, uint8_t *img, int64_t row_blocks,
                             const int32_t *live, void *ws, cudaStream_t s) {
    const Layout l = layout_of(c.Hkv, c.D, a.n_heads, B, T);
    uint8_t *w = static_cast<uint8_t *>(ws);
    const DecodeArgs p = {c, a, B, T, a.n_heads / c.Hkv, l.groups, l.tile / c.page_tokens, l.tile % c.page_tokens, live, reinterpret_cast<float *>(w + l.acc),
                          reinterpret_cast<float2 *>(w + l.ml), reinterpret_cast<int64_t *>(w + l.plan)};
    qk_status st = l.tile != TILE ? launch_attn_wide(p, l.NT, s)
                   : c.D == 256  ? launch_pass<256, 1>(p, s)
                   : c.D == 64 ? (l.NT == 1 ? launch_pass<64, 1>(p, s) : launch_pass<64, 2>(p, s))
                               : (l.NT == 1 ? launch_pass<128, 1>(p, s) : launch_pass<128, 2>(p, s));
    if (st != QK_OK) return st;
    const int rows = B * T;
    const JoinArgs j = {p, img, row_blocks, l.NT, l.tile};
    // Many heads have few partial results each: a warp a head; few heads have many: a CTA a head. Whole calls, us, by CTAs /
    // by warps: 32 heads behind 131072 keys 62 / 114, 224 behind 2000 12.7 / 18.7, 512 behind 8192 30.0 / 34.5, 1024 behind
    // 8192 42.5 / 44.7, 1792 behind 8192 67.7 / 67.2, 4096 of 1500 to 9000 keys (32 columns of 128) 78.3 / 75.0.
    const int64_t heads = (int64_t)rows * a.n_heads;
    if (heads >= 1024) {
        auto *combine = c.D == 64    ? attn_combine_warps_kernel<64>
                        : c.D == 128 ? attn_combine_warps_kernel<128>
                                     : attn_combine_warps_kernel<256>;
        return launch_pdl("attn_combine", combine, dim3((unsigned)ceil_div(heads, 4)), dim3(128), 0, s, j);
    }
    auto *combine = c.D == 64 ? attn_combine_kernel<64> : c.D == 128 ? attn_combine_kernel<128> : attn_combine_kernel<256>;
    return launch_pdl("attn_combine", combine, dim3(a.n_heads, (unsigned)rows), dim3(128), 0, s, j);
}

qk_status read_attn_decode_faults(uint32_t *faults) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tc_faults, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_tc_faults, &zero, sizeof zero);
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "qk_device_faults: %s", cudaGetErrorString(e));
    *faults = v;
    return QK_OK;
}

}  // namespace qk

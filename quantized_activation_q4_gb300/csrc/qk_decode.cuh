// What the decode attention's kernels have in common: the shares of keys, fragments of packed codes.
#pragma once

#include "qk_kv.cuh"
#include "qk_tc.cuh"

namespace qk {

struct DecodeArgs {
    KvCache c;
    qk_attn a;
    int B, T, G, groups;   // groups: CTAs that share a tile, each with its own columns
    int tile_pages, tile_rest;   // a tile / page_tokens, a tile % page_tokens
    const int32_t *live;
    float *acc;            // [slot][groups][8 NT][D]
    float2 *ml;            // [slot][groups][8 NT]: reference maximum, sum of weights
    int64_t *plan;         // [0] tiles of a share, [1 + b] tiles before sequence b
};

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float HEADROOM = 8.0f;    // the reference maximum moves when a logit is 2^8 above it
constexpr float LIFT = 6.0f;        // weights are held times 2^6 below the reference: at most 2^14
constexpr int MAX_CTAS = 1024;      // of one launch; sizes the workspace

// ---------------------------------------------------------------- the tiles of a sequence
struct Sequence {
    int len, base, tiles;   // keys, first token that a tile covers (a multiple of 16), tiles of one head
};
template <int TILE>   // tokens of a tile
__device__ __forceinline__ Sequence sequence_of(const DecodeArgs &p, int b) {
    const int64_t most = p.a.table_stride * p.c.page_tokens;
    Sequence s;
    s.len = (int)min((int64_t)max(ld_prev(p.a.kv_lens + b), 0), most);
    const int first_end = s.len - p.T + 1;
    s.base = p.a.window > 0 ? max(0, first_end - p.a.window) & ~(GROUP - 1) : 0;
    s.tiles = (s.len - s.base + TILE - 1) / TILE;   // lengths are at most 2^30
    return s;
}

// Sum over a CTA of one value a thread, and the sum of the threads before.
template <int WARPS>
__device__ __forceinline__ int64_t scan_cta(int64_t v, int64_t *before, int64_t *smem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, m);
        if (lane >= m) x += y;
    }
    __syncthreads();
    if (lane == 31) smem[warp] = x;
    __syncthreads();
    int64_t total = 0, base = 0;
#pragma unroll
    for (int w = 0; w < WARPS; w++) {
        if (w < warp) base += smem[w];
        total += smem[w];
    }
    *before = base + x - v;
    return total;
}

// A walk over the tiles of a share: (sequence, head, tile), sequences without keys left out.
struct Walk {
    int b, h, tile;
    Sequence s;
};
template <int TILE>
__device__ __forceinline__ void next_tile(Walk &w, const DecodeArgs &p, int live) {
    if (++w.tile < w.s.tiles) return;
    w.tile = 0;
    if (++w.h < p.c.Hkv) return;
    w.h = 0;
    do {
        w.b++;
        if (w.b < live) w.s = sequence_of<TILE>(p, w.b);
    } while (w.b < live && w.s.tiles == 0);
}

// The share of a CTA: its first tile and how many there are (0: none, `now` is not set). CTA 0 leaves the plan for the join.
// Of up to WARPS * 32 sequences a thread keeps its own from the one look to the other. (Lengths are loaded beside the live
// count.)
template <int WARPS, int TILE>
__device__ __forceinline__ int64_t share_of(const DecodeArgs &p, int live, int share, int shares, int64_t *scan, int64_t *found,
                                            Walk &now) {
    int64_t total = 0, before = 0, n = 0;
    const auto tiles_of = [&](int b) {
        const int tiles = b < p.B ? sequence_of<TILE>(p, b).tiles : 0;
        return b < live ? (int64_t)tiles * p.c.Hkv : 0;
    };
    for (int b0 = 0; b0 < p.B; b0 += WARPS * 32) {
        const int b = b0 + threadIdx.x;
        n = tiles_of(b);
        const int64_t sum = scan_cta<WARPS>(n, &before, scan);
        if (blockIdx.x == 0 && b < live) p.plan[1 + b] = total + before;
        total += sum;
    }
    const int64_t each = max((int64_t)1, (total + shares - 1) / shares);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.plan[0] = each;
    const int64_t first = share * each, left = min(each, total - first);
    if (left <= 0) return 0;
    int64_t at = 0;
    for (int b0 = 0; b0 < p.B; b0 += WARPS * 32) {
        const int b = b0 + threadIdx.x;
        int64_t sum = total;
        if (p.B > WARPS * 32) {
            n = tiles_of(b);
            sum = scan_cta<WARPS>(n, &before, scan);
        }
        if (first >= at + before && first < at + before + n) {
            found[0] = b;
            found[1] = first - at - before;
        }
        at += sum;
        if (first < at) break;
    }
    __syncthreads();
    now.b = (int)found[0];
    now.s = sequence_of<TILE>(p, now.b);
    now.h = (int)(found[1] / now.s.tiles);
    now.tile = (int)(found[1] % now.s.tiles);
    return left;
}

// ---------------------------------------------------------------- fragments
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(half2_bits(a), half2_bits(b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = lds32(a);
    } else if constexpr (N == 2) {
        const uint2 v = lds64(a);
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = lds128(a + 4 * i);
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    }
}


}  // namespace

// The pass for more query columns than the first kernel's (k_attn_wide.cu); tokens of its tiles.
constexpr int WIDE_TILE = 64, WIDE_COLUMNS = 4;   // column tiles of 8 a CTA takes at most
qk_status launch_attn_wide(const DecodeArgs &p, int NT, cudaStream_t s);

}  // namespace qk

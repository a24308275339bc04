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

// ---------------------------------------------------------------- sizes of the values
// The second product's operand is weight times scale in binary16, whose least step is 2^-24. `top` is the exponent of the
// largest scale seen in the segment. Weights are 2^(LIFT - lift) at the reference, scales are taken times 2^boost:
//   top        lift    boost           a key's product, next to that of the reference's weight and scale 2^top, is off by
//   below -3   0       -top            2^-31 (a product of boosted scales is exact)
//   -3 .. 6    0 .. 6  0               2^-28, less where scales are larger
//   above 6    6       6 - top         2^-31, and its weight by 2^-25
// and by 2^-10 of itself. So products stay below 2^15, and the offset of the weights is never above the reference: of huge
// logits one number holds only one of both, and weights would be lost with a higher one. Before the first key top is least.
constexpr int SMALLEST = -24, USUAL = -3;
__device__ __forceinline__ int lift_of(int top) { return min(max(top, 0), (int)LIFT); }
__device__ __forceinline__ bool usual(int top) { return top >= USUAL && top <= (int)LIFT; }
__device__ __forceinline__ int boost_of(int top) { return usual(top) ? 0 : lift_of(top) - top; }
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// The values' scales of N groups side by side in shared memory, a pair a lane and turn: `f` gets its address and the place of
// its first token. `at`: the first group's scales.
template <int NB, int N, typename F>
__device__ __forceinline__ void each_scales(uint32_t at, F f) {
    constexpr int PAIRS = 8 * NB;   // of a group
#pragma unroll
    for (int x0 = 0; x0 < N * PAIRS; x0 += 32) {
        const int x = x0 + (threadIdx.x & 31), y = x % PAIRS;
        if (N * PAIRS % 32 == 0 || x < N * PAIRS)
            f(at + x / PAIRS * group_bytes(32 * NB) + 4 * y, x / PAIRS * GROUP + y / (2 * NB) * 2 + y % 2 * 8);
    }
}
// Whether one of them is 2 or more: bit 14 of a half is set from there on. (A lane's own alone.)
template <int NB, int N>
__device__ __forceinline__ bool large_scales(uint32_t at) {
    uint32_t any = 0;
    each_scales<NB, N>(at, [&](uint32_t a, int) { any |= lds32(a); });
    return (any & 0x40004000u) != 0;
}
// The exponent of the largest one, or `least` if that is larger.
template <int NB, int N>
__device__ __forceinline__ int largest_exponent(uint32_t at, int least) {
    __half2 m = half2_bits(0);
    each_scales<NB, N>(at, [&](uint32_t a, int) { m = __hmax2(m, __habs2(half2_bits(lds32(a)))); });
#pragma unroll
    for (int x = 16; x; x >>= 1) m = __hmax2(m, __shfl_xor_sync(FULL, m, x));
    return max(least, (int)(__float_as_uint(fmaxf(__low2float(m), __high2float(m))) >> 23) - 127);
}
// Rewrites them (rarely needed, so the products' loop has nothing of it). The next copy into the stage comes after the fence.
template <int NB, int N, typename F>
__device__ __forceinline__ void rewrite_scales(uint32_t at, F to) {
    each_scales<NB, N>(at, [&](uint32_t a, int token) {
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(to(lds32(a), token)) : "memory");
    });
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}
// Zero for keys that no token sees: there the cache may hold anything. Seen are [begin, end) of the groups in `used` (a byte
// each), counted from the first group's first token.
template <int NB, int N>
__device__ __forceinline__ void hide_scales(uint32_t at, int begin, int end, uint32_t used) {
    rewrite_scales<NB, N>(at, [=](uint32_t v, int i) {
        const uint32_t seen = (i >= begin && i < end ? 0xffffu : 0) | (i + 1 >= begin && i + 1 < end ? 0xffff0000u : 0);
        return used >> (8 * (i / GROUP)) & 1 ? v & seen : 0;
    });
}
// Times 2^boost, -10..24, in two steps for what binary16 does not hold.
template <int NB, int N>
__device__ __forceinline__ void boost_scales(uint32_t at, int boost) {
    const float first = power_of_two(min(boost, 15)), rest = power_of_two(boost - min(boost, 15));
    rewrite_scales<NB, N>(at, [=](uint32_t v, int) { return mul2(mul2(v, pack2(first, first)), pack2(rest, rest)); });
}

}  // namespace

// The pass for more query columns than the first kernel's (k_attn_wide.cu); tokens of its tiles.
constexpr int WIDE_TILE = 64, WIDE_COLUMNS = 4;   // column tiles of 8 a CTA takes at most
qk_status launch_attn_wide(const DecodeArgs &p, int NT, cudaStream_t s);

}  // namespace qk

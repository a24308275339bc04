// Matrix-vector products with group-scaled 4-bit weights (QK_W_Q4_G64, QK_W_Q4_G128) on a shared
// Q8_1 image, ordinary and routed per expert: the calls of llama.cpp PR #117 (Overview, Coverage:
// MUL_MAT and MUL_MAT_ID readers of one image) for weights with a scale and a zero point per group.
//
//   y[t][n] = sum_g d[n][g] * sum_{b in g} d_a[t][b] * sum_{i in b} (nibble_i - z[n][g]) * q_i
//
// Every block sum is exact (integers); the sums over blocks and groups are binary32.

#include <atomic>
#include <cstdlib>

#include "qk_internal.cuh"

namespace qk {
namespace {

constexpr int MAX_PROJ = 8, MAX_E = 1024;
constexpr unsigned FULL = 0xffffffffu;

__device__ unsigned int g_mmvq_g_faults = 0;   // bits as qk_device_faults

// ---------------------------------------------------------------- weight pack
// One CTA per unit (32 rows x 128 columns). Source block: half d, z, unread, G/2 nibble bytes.
template <int G>
__global__ void __launch_bounds__(256) pack_g_kernel(const uint8_t *__restrict__ src, int N, int K, int chunks,
                                                     uint8_t *__restrict__ packed) {
    constexpr int SRC = 4 + G / 2, UNIT = strip_unit_bytes(G);
    const int64_t unit = blockIdx.x;
    const int64_t strip = unit / chunks;
    const int chunk = (int)(unit - strip * chunks);
    uint8_t *dst = packed + unit * UNIT;
    const int64_t row_bytes = (int64_t)(K / G) * SRC;
    for (int w = threadIdx.x; w < STRIP_DATA / 4; w += 256) {
        const int jb = w >> 7, lane = (w >> 2) & 31, i = w & 3;
        const int64_t n = strip * STRIP_ROWS + (lane >> 2) + 8 * i;
        const int col = chunk * UNIT_COLS + jb * QB;
        uint32_t v = 0;
        if (n < N && col < K) {
            const uint8_t *p = src + n * row_bytes + (int64_t)(col / G) * SRC + 4 + (col % G) / 2 + 4 * (lane & 3);
            v = (uint32_t)p[0] | ((uint32_t)p[1] << 8) | ((uint32_t)p[2] << 16) | ((uint32_t)p[3] << 24);
        }
        reinterpret_cast<uint32_t *>(dst)[w] = v;
    }
    for (int w = threadIdx.x; w < (UNIT - STRIP_DATA) / 4; w += 256) {
        const int grp = w >> 5, g = (w >> 2) & 7, i = w & 3;
        const int64_t n = strip * STRIP_ROWS + g + 8 * i;
        const int col = chunk * UNIT_COLS + grp * G;
        uint32_t v = 0;
        if (n < N && col < K) {
            const uint8_t *p = src + n * row_bytes + (int64_t)(col / G) * SRC;
            const __half z = __int2half_rn((int)(p[2] & 15) - 8);
            v = (uint32_t)p[0] | ((uint32_t)p[1] << 8) | ((uint32_t)__half_as_ushort(z) << 16);
        }
        reinterpret_cast<uint32_t *>(dst + STRIP_DATA)[w] = v;
    }
}

// ---------------------------------------------------------------- matvec
// Bound by the weight stream. A warp multiplies a strip of 32 rows by up to eight tokens with
// mma.sync m16n8k16 (weights as A, straight from global memory: the packed order is the fragment order;
// tokens as B). A nibble becomes a half by one logic operation, 1024 + c or 64 + c; the biases and the
// 8 of a middle zero point leave with the accumulator's start value, so every block sum is exact:
//   D_b = sum (c - 8) q,   group = sum_b d_a D_b,   y += d (group - (z - 8) sum_b d_a sum q)
// About 150 instructions per 32 x 128 weights, so that the 2176 bytes take as long from memory as from
// the issue slots of a quarter of the SM at half rate.
//
// A CTA turns its share of the image into B fragments in shared memory once (for every row block it then
// takes), its warps take wr = WARPS / wk strips times wk pieces of the share, and the partial sums meet in
// shared memory, added in the order of K. Work items are (pass, row block); a pass is the call's tokens, or
// up to eight planned pairs of one expert. Every CTA takes a contiguous range of items, and the loads of
// the next item's weights are in flight while one is finished. A CTA has all of K, or a cluster of `split` CTAs
// shares it and sums in distributed shared memory; the release of a cluster's barrier waits for the weight
// loads in flight, so that an item of a cluster costs about 4 us and clusters pay only for few items
// (launch_matvec has the figures).
// 8192 -> 65536, four tokens: 55 us, 5.2 TB/s. Gate/up of 13 live rows, top 8 of 128 experts, 2560 -> 2 x 768: 38 us,
// 4.2 TB/s. In both the products stream at 6 TB/s; the start and the fragments of K take 12 and 15 thousand
// cycles before them, an item's sums 1.6 thousand after.
constexpr int RED_STRIDE = 36;       // floats between two tokens' 32 rows of partial sums: no bank conflicts
constexpr int RED = 8 * RED_STRIDE;  // floats of one warp's partial sums
constexpr int FEW_WARPS = 8, MANY_WARPS = 16;
// chunks of K whose fragments a CTA holds at a time: as many as two CTAs per SM, or one, have room for
__host__ __device__ constexpr int max_chunks(int warps) { return warps == FEW_WARPS ? 34 : 72; }
constexpr int SHORT_CHUNKS = 20;     // K up to 2560
constexpr int PFD = 2;               // chunks ahead on their way into L2 (4, 8 or 16 were no faster)
constexpr uint32_t SUSPEND_NS = 20000;
constexpr int WAIT_TRIES = 1 << 16;  // a wait gives up after about a second; QK_MMVQ_G_WAIT_TRIES overrides it (tests)

struct GProj {
    const uint8_t *w;
    float *y;
    int64_t y_stride, expert_bytes;
    int N, K, chunks;
};
struct GArgs {
    const uint8_t *img;
    int64_t img_row_bytes;
    const int32_t *live, *counts, *offsets, *items;
    int T, k, E, per_pair, n_proj;   // T: tokens, or bucket rows of a routed call
    int wait_tries;                  // looks of up to SUSPEND_NS at a barrier before a wait gives up
    int wk_log2, held;               // wk = 1 << wk_log2 warps share a strip; chunks of fragments
    GProj p[MAX_PROJ];
};

// Fragments of one 128-column chunk: B (per block a 16-byte entry per lane), d_a and the start value of
// eight tokens per block, sum_b d_a sum q per group and token.
template <int G>
struct Rec {
    uint4 b[4][32];
    float4 start[4][4];              // (s, s') of tokens 2t, 2t+1, twice: an accumulator's four registers
    float da[4][8], xs[128 / G][8];
};
template <int G>
struct Chunk {
    uint4 w[4], head[128 / G];
};

__device__ __forceinline__ uint4 ldg_stream16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
template <int G>
__device__ __forceinline__ void load_chunk(Chunk<G> &c, const uint8_t *unit, int lane) {
#pragma unroll
    for (int jb = 0; jb < 4; jb++) c.w[jb] = ldg_stream16(unit + jb * 512 + lane * 16);
#pragma unroll
    for (int g = 0; g < 128 / G; g++) c.head[g] = ldg_stream16(unit + STRIP_DATA + 128 * g + 16 * (lane >> 2));
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// D = A_lo B_lo + A_hi B_hi + start for 16 rows (words w0 of row g, w1 of row g + 8) x 8 tokens
__device__ __forceinline__ void block_dot(uint32_t w0, uint32_t w1, uint4 b, float4 s, uint64_t &d01, uint64_t &d23) {
    float e0, e1, e2, e3;
    asm("{\n"
        ".reg .b32 v0, v1, l0, l1, l2, l3, h0, h1, h2, h3;\n"
        ".reg .f32 c0, c1, c2, c3;\n"
        "shr.b32 v0, %4, 8;\n"
        "shr.b32 v1, %5, 8;\n"
        "lop3.b32 l0, %4, 0x000F000F, 0x64006400, 0xEA;\n"
        "lop3.b32 l1, %5, 0x000F000F, 0x64006400, 0xEA;\n"
        "lop3.b32 l2, v0, 0x000F000F, 0x64006400, 0xEA;\n"
        "lop3.b32 l3, v1, 0x000F000F, 0x64006400, 0xEA;\n"
        "lop3.b32 h0, %4, 0x00F000F0, 0x54005400, 0xEA;\n"
        "lop3.b32 h1, %5, 0x00F000F0, 0x54005400, 0xEA;\n"
        "lop3.b32 h2, v0, 0x00F000F0, 0x54005400, 0xEA;\n"
        "lop3.b32 h3, v1, 0x00F000F0, 0x54005400, 0xEA;\n"
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {c0,c1,c2,c3}, {l0,l1,l2,l3}, {%6,%7}, {%10,%11,%12,%13};\n"
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {h0,h1,h2,h3}, {%8,%9}, {c0,c1,c2,c3};\n"
        "}\n"
        : "=f"(e0), "=f"(e1), "=f"(e2), "=f"(e3)
        : "r"(w0), "r"(w1), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w), "f"(s.x), "f"(s.y), "f"(s.z),
          "f"(s.w));
    d01 = pack2(e0, e1);
    d23 = pack2(e2, e3);
}

// y (rows g, g+8, 16+g, 24+g of the strip x tokens 2t, 2t+1) += the chunk's products
template <int G>
__device__ __forceinline__ void chunk_product(const Chunk<G> &c, const Rec<G> &r, int lane, uint64_t y[4]) {
    constexpr int BG = G / 32;   // blocks per group
    const int t2 = 2 * (lane & 3);
#pragma unroll
    for (int grp = 0; grp < 128 / G; grp++) {
        uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < BG; i++) {
            const int jb = grp * BG + i;
            const uint4 b = r.b[jb][lane];
            const float2 da = *reinterpret_cast<const float2 *>(&r.da[jb][t2]);
            const float4 st = r.start[jb][lane & 3];
            const uint64_t da2 = pack2(da.x, da.y);
            uint64_t d01, d23;
            block_dot(c.w[jb].x, c.w[jb].y, b, st, d01, d23);
            acc[0] = fma2(da2, d01, acc[0]);
            acc[1] = fma2(da2, d23, acc[1]);
            block_dot(c.w[jb].z, c.w[jb].w, b, st, d01, d23);
            acc[2] = fma2(da2, d01, acc[2]);
            acc[3] = fma2(da2, d23, acc[3]);
        }
        const float2 xs = *reinterpret_cast<const float2 *>(&r.xs[grp][t2]);
        const uint64_t xs2 = pack2(xs.x, xs.y);
        const uint32_t h[4] = {c.head[grp].x, c.head[grp].y, c.head[grp].z, c.head[grp].w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 dz = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));   // d, z - 8
            y[i] = fma2(pack2(dz.x, dz.x), fma2(pack2(-dz.y, -dz.y), xs2, acc[i]), y[i]);
        }
    }
}

// A warp's fragments of one chunk: lane (g, t) converts words t of token g's blocks. Columns past K and
// absent tokens (no row) are zeros; nothing of them is read. Loads and conversion apart, so that several
// chunks' loads are in flight at once.
struct Words {
    uint32_t lo[4], hi[4], ds;   // ds: the head of block t
};
__device__ __forceinline__ void load_words(Words &w, const uint8_t *img_row, int chunk, int K, int lane) {
    const int t = lane & 3;
    w.ds = 0;
#pragma unroll
    for (int jb = 0; jb < 4; jb++) {
        w.lo[jb] = w.hi[jb] = 0;
        if (img_row && chunk * UNIT_COLS + jb * QB < K) {
            const uint8_t *blk = img_row + (int64_t)(4 * chunk + jb) * Q8_1_BYTES;
            w.lo[jb] = ld_prev(reinterpret_cast<const uint32_t *>(blk + 4 + 4 * t));
            w.hi[jb] = ld_prev(reinterpret_cast<const uint32_t *>(blk + 20 + 4 * t));
        }
    }
    if (img_row && chunk * UNIT_COLS + t * QB < K)
        w.ds = ld_prev(reinterpret_cast<const uint32_t *>(img_row + (int64_t)(4 * chunk + t) * Q8_1_BYTES));
}
template <int G>
__device__ __forceinline__ void make_rec(Rec<G> &r, const Words &w, int lane) {
    const int g = lane >> 2, t = lane & 3;
    int sums[4];   // of a block's low and high halves, 16 bits each (|sum| <= 16 * 128)
#pragma unroll
    for (int jb = 0; jb < 4; jb++) {
        // codes -> exact halves: q + 128 under the exponent of 1024, minus 1152
        const uint32_t u = w.lo[jb] ^ 0x80808080u, v = w.hi[jb] ^ 0x80808080u;
        const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        const uint32_t p[4] = {__byte_perm(u, 0x64646464u, 0x4240), __byte_perm(u, 0x64646464u, 0x4341),
                               __byte_perm(v, 0x64646464u, 0x4240), __byte_perm(v, 0x64646464u, 0x4341)};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&p[i]), bias);
            o[i] = *reinterpret_cast<const uint32_t *>(&x);
        }
        r.b[jb][lane] = make_uint4(o[0], o[1], o[2], o[3]);
        sums[jb] = __dp4a((int)w.lo[jb], 0x01010101, 0) + (__dp4a((int)w.hi[jb], 0x01010101, 0) << 16);
    }
    // four lanes' sums of four blocks, in three shuffles: lane t ends with block t's
    const bool odd = t & 1, high = t & 2;
    int s0 = odd ? sums[1] : sums[0], s1 = odd ? sums[3] : sums[2];
    s0 += __shfl_xor_sync(FULL, odd ? sums[0] : sums[1], 1);
    s1 += __shfl_xor_sync(FULL, odd ? sums[2] : sums[3], 1);
    const int s = (high ? s1 : s0) + __shfl_xor_sync(FULL, high ? s0 : s1, 2);
    const int sl = (short)s, sh = (s - sl) >> 16;
    const float da = __half2float(__ushort_as_half((unsigned short)w.ds));
    r.da[t][g] = da;
    float *st = reinterpret_cast<float *>(&r.start[t][g >> 1]) + (g & 1);
    st[0] = st[2] = -(float)((1024 + 8) * sl + (64 + 8) * sh);
    float xs = da * (float)(sl + sh);
    xs += __shfl_xor_sync(FULL, xs, 1);
    if (G == 128) xs += __shfl_xor_sync(FULL, xs, 2);
    if (t % (G / QB) == 0) r.xs[t * QB / G][g] = xs;
}

// Pass q of a routed call: its expert and the position of its first pair among the expert's.
__device__ __forceinline__ void find_pass(const int *pre, int E, int q, int &e, int &first) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= q)
            lo = mid;
        else
            hi = mid;
    }
    e = lo;
    first = 8 * (q - pre[lo]);
}
__device__ __forceinline__ int clamped_count(const GArgs &a, int e) {
    const int c = ld_prev(a.counts + e), pairs = a.T * a.k;
    return c < 0 ? 0 : (c > pairs ? pairs : c);
}

template <int WARPS>
__host__ __device__ inline int row_blocks_of(int N, int wk_log2) {
    const int strips = (N + STRIP_ROWS - 1) / STRIP_ROWS, wr_log2 = (WARPS == FEW_WARPS ? 3 : 4) - wk_log2;
    return (strips + (1 << wr_log2) - 1) >> wr_log2;
}
// Whether 2 << wk_log2 warps may share a strip: there are so many, and each has two chunks of K.
template <int WARPS>
bool more_wk(const GArgs &a, int wk_log2) {
    return (WARPS >> wk_log2) > 1 && (a.held >> (wk_log2 + 1)) >= 2;
}
template <int WARPS>
int64_t row_blocks_of_all(const GArgs &a, int wk_log2) {
    int64_t rbs = 0;
    for (int j = 0; j < a.n_proj; j++) rbs += row_blocks_of<WARPS>(a.p[j].N, wk_log2);
    return rbs;
}
// Ordinary calls: warps over rows; over K as well (two, four.. to a strip) while that leaves CTAs without work or the
// last round of items more than a tenth empty.
template <int WARPS>
int choose_wk(const GArgs &a, int64_t clusters) {
    int wk = 0;
    for (; more_wk<WARPS>(a, wk); wk++) {
        const int64_t items = row_blocks_of_all<WARPS>(a, wk), rounds = ceil_div(items, clusters);
        if (items >= clusters && rounds * clusters * 10 <= items * 11) break;
    }
    return wk;
}
// Routed calls: the split of K decides the order of a pair's sums, so it goes by the sizes and k alone and not by the
// passes there are, which follow the live count, the bucket and other rows' routes. Many warps to a strip serve one
// token, few serve many passes: the fewest whose items at one row (k passes) reach half of the resident CTAs.
// us at 1, 2, 4, 8 warps to a strip, * the choice, and last by the passes there are with the rule for ordinary calls:
//   2560 -> 2 x 768, 8 of 128 experts:   1 row 24, 16, 12.1*, 14.3 (14.8); 4 rows 25, 23, 22.0*, 26 (26.6);
//                                        16 rows 38.8, 38.5, 39.3*, 47 (42.0); 64 rows 65, 62, 69*, 84 (65.2)
//   768 -> 2560, 8 of 128:               1 row 12.0, 9.4* (9.6); 16 rows 26.0, 27.6* (28.2); 64 rows 42, 47* (47)
//   4096 -> 512, 2 of 8:                 1 row 30, 18.5, 12.7, 9.6, 7.6 with sixteen* (8.2)
//   4096 -> 2 x 14336, 2 of 8:           1 row 33.9*, 36, 33, 36 (33.1); 8 rows 81*, 85, 89, 100 (81)
//   7168 -> 2 x 2048, 8 of 256:          1 row 52 with one, 31.9* (43); 8 rows 147, 150* (146)
//   14336 -> 4096 (slots), 2 of 8:       1 row 50, 30, 20.4* (31); 8 rows 53, 48, 45*, 53 (60)
template <int WARPS>
int choose_routed_wk(const GArgs &a, int64_t clusters) {
    int wk = 0;
    while (more_wk<WARPS>(a, wk) && 2 * a.k * row_blocks_of_all<WARPS>(a, wk) < clusters) wk++;
    return wk;
}
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int G, bool ROUTED, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) mmvq_g_kernel(const __grid_constant__ GArgs a) {
    constexpr int THREADS = WARPS * 32, MAXC = max_chunks(WARPS);
    constexpr int FLIGHT = WARPS == FEW_WARPS ? 8 : 2;   // remote loads; sixteen warps have no registers for more
    // chunks of the image in flight (two / three: routed gate/up of 16 rows 44.8 / 42.2 us, of 64 rows 68 / 65,
    // output head 55.6 / 58.7)
    constexpr int AHEAD = ROUTED || WARPS == FEW_WARPS ? 3 : 2;
    extern __shared__ __align__(16) uint8_t smem[];
    Rec<G> *rec = reinterpret_cast<Rec<G> *>(smem);
    float *red = reinterpret_cast<float *>(rec + a.held);   // [2][WARPS][RED]
    int *pre = reinterpret_cast<int *>(red + 2 * WARPS * RED);    // [E + 1], routed calls
    __shared__ __align__(8) uint64_t written;   // a CTA that sums alone: its warps' arrivals, item after item
    __shared__ int gave_up;   // a warp's wait has run out
    __shared__ int tok_row[2][8], tok_out[4][8], warp_passes[WARPS], n_pass, share_lo[MAX_PROJ], share_hi[MAX_PROJ], rb_base[MAX_PROJ + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank, split;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const int clusters = gridDim.x / split, cluster = blockIdx.x / split;
    pdl_trigger();
    const uint32_t bar = (uint32_t)__cvta_generic_to_shared(&written);
    if (threadIdx.x == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(WARPS) : "memory");
        gave_up = 0;
    }
    if (threadIdx.x < a.n_proj) {   // this CTA's chunks of K (chunks < 2^24)
        const uint32_t n = a.p[threadIdx.x].chunks;
        share_lo[threadIdx.x] = n * rank / split;
        share_hi[threadIdx.x] = n * (rank + 1) / split;
    }

    int passes = 1;
    if (ROUTED) {
        pdl_wait();   // the plan decides which weights are read
        // Prefix of the experts' passes: a thread has PER experts in a row. No plan of this bucket has more
        // than pairs / 8 + E passes; sums stop one above (counts with more: no work).
        constexpr int PER = MAX_E / THREADS;
        const int most = a.T * a.k / 8 + a.E, e0 = threadIdx.x * PER;
        int n[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; i++) n[i] = e0 + i < a.E ? (clamped_count(a, e0 + i) + 7) / 8 : 0;
#pragma unroll
        for (int i = 0; i < PER; i++) sum = min(sum + n[i], most + 1);
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl = min(incl + v, most + 1);
        }
        if (lane == 31) warp_passes[warp] = incl;
        __syncthreads();
        int total = 0, at = 0;
#pragma unroll
        for (int w = 0; w < WARPS; w++) {
            if (w == warp) at = total;
            total = min(total + warp_passes[w], most + 1);
        }
        at += incl - sum;
        const bool sound = total <= most;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            if (e0 + i < a.E) pre[e0 + i] = sound ? at : 0;
            at += n[i];
        }
        if (threadIdx.x == 0) {
            pre[a.E] = n_pass = sound ? total : 0;
            if (!sound) atomicOr(&g_mmvq_g_faults, 2u);
        }
    }
    __syncthreads();
    const int wk_log2 = a.wk_log2;
    if (ROUTED) passes = n_pass;
    if (threadIdx.x == 0) {
        int rbs = 0;
        for (int j = 0; j < a.n_proj; j++) {
            rb_base[j] = rbs;
            rbs += row_blocks_of<WARPS>(a.p[j].N, wk_log2);
        }
        rb_base[a.n_proj] = rbs;
    }
    __syncthreads();
    const int row_blocks = rb_base[a.n_proj];
    const int wk = 1 << wk_log2, wr = WARPS >> wk_log2, kw = warp & (wk - 1), ws = warp >> wk_log2;
    // this cluster's items [it0, it1)
    const uint32_t items = (uint32_t)passes * row_blocks, per = items / clusters, more = items % clusters;
    const int it0 = per * cluster + min((uint32_t)cluster, more), it1 = it0 + per + ((uint32_t)cluster < more ? 1 : 0);

    // Items are walked by additions: a place is a pass and one of its row blocks. Row block -> projection and
    // row block of the projection.
    auto proj_of = [&](int at, int &rb) {
        int j = 0;
        while (j + 1 < a.n_proj && at >= rb_base[j + 1]) j++;
        rb = at - rb_base[j];
        return j;
    };
    const int pass0 = ROUTED && it0 < it1 ? it0 / row_blocks : 0, at0 = it0 - pass0 * row_blocks;
    auto next_place = [&](int &pass, int &at) {
        if (++at == row_blocks) {
            at = 0;
            pass++;
        }
    };
    // The walk of this warp over its weights: the chunks of its strip and its piece of K, item after item,
    // sub-share (MAXC chunks) after sub-share.
    const uint8_t *wp = nullptr;
    int w_left = 0, w_items = it1 - it0 + 1, w_from = 0, w_to = 0;   // w_from .. w_to: the CTA's chunks not yet walked
    int w_pass = pass0, w_at = at0 - 1;
    auto seek = [&]() {   // to the next non-empty run; no items left at the end
        while (w_left == 0 && w_items > 0) {
            if (w_from >= w_to) {
                if (--w_items == 0) return;
                next_place(w_pass, w_at);
                w_from = w_to = 0;
            }
            int rb;
            const int j = proj_of(w_at, rb);
            const GProj &P = a.p[j];
            if (w_to == 0) {
                w_from = share_lo[j];
                w_to = share_hi[j];
            }
            int e = 0, first = 0;
            if (ROUTED) find_pass(pre, a.E, w_pass, e, first);
            const int strip = rb * wr + ws, n = min(w_to - w_from, MAXC);
            const int b = w_from + ((n * kw) >> wk_log2), end = w_from + ((n * (kw + 1)) >> wk_log2);
            w_from += n;
            if (strip * STRIP_ROWS >= P.N) continue;
            w_left = end - b;
            wp = P.w + e * P.expert_bytes + ((int64_t)strip * P.chunks + b) * strip_unit_bytes(G);
        }
    };
    auto fetch = [&](Chunk<G> &c) {
        if (w_left == 0) seek();
        if (w_left > 0) {
            // the run's chunk PFD further on, on its way into L2 without registers
            if (w_left > PFD && lane * 128 < strip_unit_bytes(G))
                asm volatile("prefetch.global.L2 [%0];" ::"l"(wp + PFD * strip_unit_bytes(G) + lane * 128));
            load_chunk<G>(c, wp, lane);
            wp += strip_unit_bytes(G);
            w_left--;
        }
    };
    Chunk<G> even, odd;   // the next two chunks of the walk; `turn`: which comes first
    int turn = 0;
    bool streaming = !ROUTED;
    if (!ROUTED) {
        fetch(even);
        fetch(odd);
        pdl_wait();   // weights are never written by the kernel before (see the header); the image may be
    }

    // Pass q's tokens: image rows and output rows, -1 for none (of a warp: its first eight lanes)
    auto list_tokens = [&](int q) {
        if (lane >= 8 || q >= passes) return;
        int row = -1, out = -1;
        if (ROUTED) {
            int e, first;
            find_pass(pre, a.E, q, e, first);
            const int64_t pos = (int64_t)ld_prev(a.offsets + e) + first + lane;
            const int pairs = a.T * a.k;
            if (first + lane < clamped_count(a, e) && pos >= 0 && pos < pairs) {
                const int pr = ld_prev(a.items + pos);
                if (pr >= 0 && pr < pairs) {
                    out = pr;
                    row = a.per_pair ? pr : pr / a.k;
                }
            }
        } else if (lane < live_rows(a.live, a.T)) {
            row = out = lane;
        }
        tok_row[q & 1][lane] = row;
        tok_out[q & 3][lane] = out;
    };
    auto announce = [&]() {
        if (split > 1) {
            cluster_arrive();
        } else {
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
        }
    };
    // The n-th announcement of every warp (of the cluster). False when it did not come, and from then on for every
    // warp: none sums, stores or announces any more, they walk through the items left only for the barriers around the
    // fragments. Nothing is stored that was not summed in full.
    auto await_sums = [&](int n) {
        if (split > 1) {
            cluster_wait();
            return true;
        }
        for (int i = 0; i < a.wait_tries; i++) {
            const int stop = *const_cast<volatile int *>(&gave_up);
            uint32_t ok;
            asm volatile(
                "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(ok)
                : "r"(bar), "r"(n & 1), "r"(SUSPEND_NS)
                : "memory");
            if (__all_sync(FULL, ok && !stop)) return true;
            if (__any_sync(FULL, stop)) break;
        }
        if (lane == 0) {
            atomicOr(&g_mmvq_g_faults, 1u);
            *const_cast<volatile int *>(&gave_up) = 1;
        }
        __syncwarp();
        return false;
    };
    // An item's sums over wk and over the cluster, in the order of K: the wr strips' 256 each, spread over
    // the cluster's threads; rows run fastest.
    auto sum_item = [&](int it, int pass, int at) {
        int rb;
        const GProj &P = a.p[proj_of(at, rb)];
        const float *base = red + (it & 1) * WARPS * RED;
        for (int v = rank * THREADS + threadIdx.x; v < wr * 256; v += split * THREADS) {
            const int s = v >> 8, tok = (v >> 5) & 7, r = v & 31, n = (rb * wr + s) * STRIP_ROWS + r;
            const int o = tok_out[pass & 3][tok];
            if (n >= P.N || o < 0) continue;
            const float *part = base + s * wk * RED + tok * RED_STRIDE + r;
            float sum = 0.0f;
            if (split == 1) {
#pragma unroll 4
                for (int w = 0; w < wk; w++) sum += part[w * RED];
            } else {   // several loads in flight: one after another 64 of them took 8 us
                const uint32_t own = (uint32_t)__cvta_generic_to_shared(part);
                const int parts = split << wk_log2;
#pragma unroll 1
                for (int i0 = 0; i0 < parts; i0 += FLIGHT) {
                    float x[FLIGHT];
#pragma unroll
                    for (int i = 0; i < FLIGHT; i++) {
                        x[i] = 0.0f;
                        if (i0 + i >= parts) continue;
                        uint32_t far;
                        asm("mapa.shared::cluster.u32 %0, %1, %2;"
                            : "=r"(far)
                            : "r"(own + 4u * ((i0 + i) & (wk - 1)) * RED), "r"((i0 + i) >> wk_log2));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[i]) : "r"(far) : "memory");
                    }
#pragma unroll
                    for (int i = 0; i < FLIGHT; i++) sum += x[i];
                }
            }
            P.y[o * P.y_stride + n] = sum;
        }
    };
    int cur_pass = -1, cur_s0 = -1, cur_cols = -1, pass = pass0, at = at0, last_pass = 0, last_at = 0;
    if (warp == WARPS - 1 && it0 < it1) list_tokens(pass0);   // the first item's syncs follow
    for (int it = it0; it < it1; it++) {
        int rb;
        const int j = proj_of(at, rb);
        const GProj &P = a.p[j];
        const bool new_pass = pass != cur_pass;
        if (new_pass) {
            cur_pass = pass;
            cur_s0 = -1;   // no fragments of this pass yet; its first items may have no share of K here
        }
        uint64_t y[4] = {0, 0, 0, 0};
        const bool mine = (rb * wr + ws) * STRIP_ROWS < P.N;
        const int c_hi = share_hi[j];
        for (int s0 = share_lo[j]; s0 < c_hi; s0 += MAXC) {
            const int s1 = min(c_hi, s0 + MAXC), cols = min(P.K, s1 * UNIT_COLS);
            if (s0 != cur_s0 || cols != cur_cols) {   // other tokens or columns than the fragments hold
                __syncthreads();   // every warp is done with the fragments before; the pass's tokens are listed
                const int row = tok_row[pass & 1][lane >> 2];
                const uint8_t *img_row = row < 0 ? nullptr : a.img + row * a.img_row_bytes;
#pragma unroll 1
                for (int c = s0 + warp;; c += AHEAD * WARPS) {
                    Words w[AHEAD];
#pragma unroll
                    for (int i = 0; i < AHEAD; i++)
                        load_words(w[i], c + i * WARPS < s1 ? img_row : nullptr, c + i * WARPS, P.K, lane);
                    if (ROUTED && !streaming) {   // behind the image's words, which are waited for first
                        streaming = true;
                        fetch(even);
                        fetch(odd);
                    }
#pragma unroll
                    for (int i = 0; i < AHEAD; i++)
                        if (c + i * WARPS < s1) make_rec<G>(rec[c + i * WARPS - s0], w[i], lane);
                    if (c + AHEAD * WARPS >= s1) break;
                }
                __syncthreads();
                cur_s0 = s0;
                cur_cols = cols;
            }
            if (!mine) continue;
            const Rec<G> *r = rec + (((s1 - s0) * kw) >> wk_log2);
            const Rec<G> *end = rec + (((s1 - s0) * (kw + 1)) >> wk_log2);
#pragma unroll 1
            while (r < end) {   // each chunk's registers are refilled as soon as they are used
                if (turn == 0) {
                    chunk_product<G>(even, *r++, lane, y);
                    fetch(even);
                    turn = 1;
                    if (r >= end) break;
                }
                chunk_product<G>(odd, *r++, lane, y);
                fetch(odd);
                turn = 0;
            }
        }
        // The next pass's tokens, after the first item of this one: the rows of the pass before have been read
        // (its fragments are made), the outputs of the one before are in another place of four.
        if (ROUTED && new_pass && warp == WARPS - 1) list_tokens(pass + 1);
        // Warps announce an item's partial sums and wait for the others' an item later, so that none stands
        // still for the slowest. When the wait for item it - 1 is over, item it - 2 has been summed by all,
        // and its buffer may be written.
        const bool go = it == it0 || await_sums(it - 1 - it0);
        if (it > it0 && go) sum_item(it - 1, last_pass, last_at);
        last_pass = pass;
        last_at = at;
        if (go) {
            float *out = red + (it & 1) * WARPS * RED + warp * RED;   // [token][32 rows]
            const int g = lane >> 2, t2 = 2 * (lane & 3);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float v0, v1;
                unpack2(y[i], v0, v1);
                out[t2 * RED_STRIDE + g + 8 * i] = v0;
                out[(t2 + 1) * RED_STRIDE + g + 8 * i] = v1;
            }
            announce();
        }
        next_place(pass, at);
    }
    if (it1 > it0) {
        if (await_sums(it1 - 1 - it0)) sum_item(it1 - 1, last_pass, last_at);
        if (split > 1) {   // no CTA leaves while another may read its sums
            cluster_arrive();
            cluster_wait();
        }
    }
}

template <typename Proj>
void fill(GArgs &a, const uint8_t *img, int64_t row_blocks, int n_proj, const Proj *projs) {
    static const int wait_tries = [] {
        const char *e = getenv("QK_MMVQ_G_WAIT_TRIES");
        return e ? atoi(e) : WAIT_TRIES;
    }();
    a.img = img;
    a.img_row_bytes = row_blocks * Q8_1_BYTES;
    a.n_proj = n_proj;
    a.wait_tries = wait_tries;
    for (int j = 0; j < n_proj; j++) {
        GProj &p = a.p[j];
        p.w = static_cast<const uint8_t *>(projs[j].w);
        p.y = projs[j].y;
        p.N = (int)projs[j].N;
        p.K = (int)projs[j].K;
        p.y_stride = p.N;
        p.chunks = (int)ceil_div(p.K, UNIT_COLS);
        p.expert_bytes = packed_bytes(projs[j].wtype, p.N, p.K);
    }
}

template <int G, bool ROUTED, int WARPS>
constexpr size_t most_smem() {   // whatever the sizes, the same CTAs fit an SM
    return max_chunks(WARPS) * sizeof(Rec<G>) + 2 * WARPS * RED * sizeof(float) + (ROUTED ? (MAX_E + 1) * 4 : 0);
}

// Clusters of `split` CTAs that are resident at once, per device (0: the query failed).
template <int G, bool ROUTED, int WARPS>
int resident_clusters(int split) {
    constexpr int MAXDEV = 64;
    static std::atomic<int> cache[MAXDEV][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAXDEV) return 0;
    int n = cache[dev][split].load(std::memory_order_relaxed);
    if (n == 0) {
        constexpr size_t smem = most_smem<G, ROUTED, WARPS>();
        static_assert(16 / WARPS * (smem + 2048) <= 227 * 1024, "shared memory");
        auto kernel = mmvq_g_kernel<G, ROUTED, WARPS>;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3(split * 64);
        cfg.blockDim = dim3(WARPS * 32);
        cfg.dynamicSmemBytes = smem;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = split;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
        cache[dev][split].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int G, bool ROUTED, int WARPS>
qk_status launch_form(GArgs &a, int64_t passes, int split, int chunks, cudaStream_t s) {
    const int64_t resident = resident_clusters<G, ROUTED, WARPS>(split);
    if (resident < 1) return fail(QK_ERR_CUDA, "mmvq: no cluster of %d CTAs fits", split);
    const int share = (int)ceil_div(chunks, split);
    a.held = share < max_chunks(WARPS) ? share : max_chunks(WARPS);
    a.wk_log2 = ROUTED ? choose_routed_wk<WARPS>(a, resident) : choose_wk<WARPS>(a, resident);
    const int64_t items = passes * row_blocks_of_all<WARPS>(a, a.wk_log2);   // fit an int (qk_api.cu)
    const int clusters = (int)(items < resident ? items : resident);
    const size_t smem = a.held * sizeof(Rec<G>) + 2 * WARPS * RED * sizeof(float) + (ROUTED ? (a.E + 1) * 4 : 0);
    auto kernel = mmvq_g_kernel<G, ROUTED, WARPS>;
    constexpr int THREADS = WARPS * 32;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)(clusters * split));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    count_launch();
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "mmvq: %s", cudaGetErrorString(e));
    return check_launch("mmvq");
}

// passes: at most this many.
template <int G, bool ROUTED>
qk_status launch_matvec(GArgs &a, int64_t passes, cudaStream_t s) {
    int chunks = 0;
    for (int j = 0; j < a.n_proj; j++) chunks = a.p[j].chunks > chunks ? a.p[j].chunks : chunks;
    // Which form (us for eight warps alone / sixteen alone / clusters of up to eight CTAs, T = 4):
    //   short K, fragments made soon: eight warps, two CTAs per SM. 1024 -> 4096: 4.3 / 4.8 / 5.2, 2560 -> 512:
    //     5.4 / 5.8 / 5.7, 2560 -> 16384: 10.7 / 10.7 / 12.9.
    //   fewer than two units for every warp of the GPU: K shared by the most CTAs (up to 8) whose equal shares
    //     waste at most a tenth. 4096 -> 512: 6.6 / 6.0 / 5.1, 8192 -> 2048: 12.5 / 9.6 / 7.2.
    //   else sixteen warps, and K shared only as far as its fragments do not fit one CTA: 8192 -> 4096:
    //     17 / 10.2 / 12.4, 8192 -> 16384: 35 / 24 / 38; 18944 -> 16384 in clusters of 1, 2, 3, 4, 8 CTAs of
    //     sixteen: 84, 84, 43, 75, 60 (one and two make fragments for every item anew).
    // A routed call never shares K for want of units: a pair's sums would be added in another order where the bucket
    // has more rows. Sixteen warps to a strip do as well (4096 -> 512, 2 of 8, 1 row: 8.2 in clusters, 7.6).
    // Routed calls with eight or sixteen warps where eight would hold K's 21 to 34 chunks too: 2688 -> 2 x 1408, 4 of
    // 60, 8 rows 28.2 / 28.1; 4096 -> 2 x 1536, 2 of 8, 4 rows 18.0 / 17.0; 4096 -> 2 x 14336, 2 of 8, 8 rows 88 / 81.
    int64_t units = 0;
    for (int j = 0; j < a.n_proj; j++) units += ceil_div(a.p[j].N, STRIP_ROWS) * a.p[j].chunks;
    if (chunks <= SHORT_CHUNKS) return launch_form<G, ROUTED, FEW_WARPS>(a, passes, 1, chunks, s);
    if (!ROUTED && units < 2 * MANY_WARPS * sm_count()) {
        int split = 1;
        for (int q = 2; q <= 8 && q <= chunks; q++)
            if (ceil_div(chunks, q) * q * 10 <= (int64_t)chunks * 11) split = q;
        return launch_form<G, ROUTED, FEW_WARPS>(a, passes, split, chunks, s);
    }
    const int64_t split = ceil_div(chunks, max_chunks(MANY_WARPS));
    return launch_form<G, ROUTED, MANY_WARPS>(a, passes, (int)(split < 8 ? split : 8), chunks, s);
}

}  // namespace

qk_status launch_weight_pack_g(int wtype, const uint8_t *blocks, int64_t N, int64_t K, uint8_t *packed,
                               cudaStream_t s) {
    const int64_t chunks = ceil_div(K, UNIT_COLS), units = ceil_div(N, STRIP_ROWS) * chunks;
    if (units > INT32_MAX) return fail(QK_ERR_UNSUPPORTED, "weight_pack: too many units for one launch");
    if (wtype == QK_W_Q4_G64)
        pack_g_kernel<64><<<(unsigned)units, 256, 0, s>>>(blocks, (int)N, (int)K, (int)chunks, packed);
    else
        pack_g_kernel<128><<<(unsigned)units, 256, 0, s>>>(blocks, (int)N, (int)K, (int)chunks, packed);
    count_launch();
    return check_launch("weight_pack");
}

qk_status launch_mmvq_g(const uint8_t *img, int64_t row_blocks, int T, int n_proj, const qk_proj *projs,
                        const int32_t *live, cudaStream_t s) {
    GArgs a = {};
    fill(a, img, row_blocks, n_proj, projs);
    for (int j = 0; j < n_proj; j++) a.p[j].y_stride = projs[j].y_stride;
    a.T = T;
    a.live = live;
    return projs[0].wtype == QK_W_Q4_G64 ? launch_matvec<64, false>(a, 1, s) : launch_matvec<128, false>(a, 1, s);
}

qk_status launch_mmvq_g_id(const uint8_t *img, int64_t row_blocks, int rows, int k, int n_proj,
                           const qk_proj_id *projs, const int32_t *counts, const int32_t *offsets,
                           const int32_t *items, bool per_pair, cudaStream_t s) {
    GArgs a = {};
    fill(a, img, row_blocks, n_proj, projs);
    a.T = rows;
    a.k = k;
    a.E = projs[0].n_experts;
    a.per_pair = per_pair;
    a.counts = counts;
    a.offsets = offsets;
    a.items = items;
    const int64_t pairs = (int64_t)rows * k, passes = pairs < pairs / 8 + a.E ? pairs : pairs / 8 + a.E;
    return projs[0].wtype == QK_W_Q4_G64 ? launch_matvec<64, true>(a, passes, s) : launch_matvec<128, true>(a, passes, s);
}

qk_status read_mmvq_g_faults(uint32_t *faults) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_mmvq_g_faults, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_mmvq_g_faults, &zero, sizeof zero);
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "qk_device_faults: %s", cudaGetErrorString(e));
    *faults = v;
    return QK_OK;
}

}  // namespace qk

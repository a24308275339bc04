// Matrix-vector products with group-scaled 4-bit weights (QK_W_Q4_G64, QK_W_Q4_G128) on a shared
// Q8_1 image, ordinary and routed per expert: the calls of llama.cpp PR #117 (Overview, Coverage:
// MUL_MAT and MUL_MAT_ID readers of one image) for weights with a scale and a zero point per group.
//
//   y[t][n] = sum_g d[n][g] * sum_{b in g} d_a[t][b] * sum_{i in b} (nibble_i - z[n][g]) * q_i
//
// Every block sum is exact (integers); the sums over blocks and groups are binary32.

#include "qk_internal.cuh"

namespace qk {
namespace {

constexpr int MAX_PROJ = 8;
constexpr unsigned FULL = 0xffffffffu;

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
struct GProj {
    const uint8_t *w;
    float *y;
    int64_t y_stride, expert_bytes;
    int N, K, chunks, strip_base;   // strip_base: first strip of this projection in the launch
};
struct GArgs {
    const uint8_t *img;
    int64_t img_row_bytes;
    const int32_t *live, *counts, *offsets, *items;
    int T, k, E, per_pair, n_proj;
    GProj p[MAX_PROJ];
};

// One row n of one projection against one image row: lane l takes blocks l, l + 32, ...
template <int G>
__device__ float row_dot(const uint8_t *w, int chunks, int K, int n, const uint8_t *img, int lane) {
    constexpr int UNIT = strip_unit_bytes(G);
    const int r = n % STRIP_ROWS, g = r & 7, i = r >> 3;
    const uint8_t *strip = w + (int64_t)(n / STRIP_ROWS) * chunks * UNIT;
    float acc = 0.0f;
    for (int b = lane; b < K / QB; b += 32) {
        const uint8_t *unit = strip + (int64_t)(b >> 2) * UNIT;
        const uint32_t head = *reinterpret_cast<const uint32_t *>(unit + STRIP_DATA + 128 * ((b & 3) * QB / G) +
                                                                  16 * g + 4 * i);
        const int z = 8 + (int)__half2float(__ushort_as_half((unsigned short)(head >> 16)));
        const uint8_t *blk = img + (int64_t)b * Q8_1_BYTES;
        const int8_t *q = reinterpret_cast<const int8_t *>(blk + 4);
        int D = 0;
        for (int t = 0; t < 4; t++) {
            const uint32_t v = *reinterpret_cast<const uint32_t *>(unit + (b & 3) * 512 + (4 * g + t) * 16 + 4 * i);
            for (int j = 0; j < 4; j++) {
                D += ((int)((v >> (8 * j)) & 15) - z) * q[4 * t + j];
                D += ((int)((v >> (8 * j + 4)) & 15) - z) * q[16 + 4 * t + j];
            }
        }
        const float da = __half2float(*reinterpret_cast<const __half *>(blk));
        acc = fmaf(__half2float(__ushort_as_half((unsigned short)head)), da * (float)D, acc);
    }
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(FULL, acc, o);
    return acc;
}

// grid (strips of every projection), 8 warps; warp w takes rows w, w + 8, ... of the strip.
template <int G>
__global__ void __launch_bounds__(256) mmvq_g_kernel(const __grid_constant__ GArgs a) {
    pdl_trigger();
    pdl_wait();
    int j = 0;
    while (j + 1 < a.n_proj && (int)blockIdx.x >= a.p[j + 1].strip_base) j++;
    const GProj &P = a.p[j];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, live = live_rows(a.live, a.T);
    for (int r = warp; r < STRIP_ROWS; r += 8) {
        const int n = ((int)blockIdx.x - P.strip_base) * STRIP_ROWS + r;
        if (n >= P.N) break;
        for (int t = 0; t < live; t++) {
            const float v = row_dot<G>(P.w, P.chunks, P.K, n, a.img + t * a.img_row_bytes, lane);
            if (lane == 0) P.y[t * P.y_stride + n] = v;
        }
    }
}

// grid (strips of every projection, experts); the pairs of the expert one after another.
template <int G>
__global__ void __launch_bounds__(256) mmvq_g_id_kernel(const __grid_constant__ GArgs a) {
    pdl_trigger();
    pdl_wait();
    int j = 0;
    while (j + 1 < a.n_proj && (int)blockIdx.x >= a.p[j + 1].strip_base) j++;
    const GProj &P = a.p[j];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y, pairs = a.T * a.k;
    const int cnt = min(max(a.counts[e], 0), pairs);
    const int64_t first = a.offsets[e];
    for (int r = warp; r < STRIP_ROWS; r += 8) {
        const int n = ((int)blockIdx.x - P.strip_base) * STRIP_ROWS + r;
        if (n >= P.N) break;
        for (int c = 0; c < cnt; c++) {
            const int64_t pos = first + c;
            if (pos < 0 || pos >= pairs) continue;
            const int p = a.items[pos];
            if (p < 0 || p >= pairs) continue;
            const int row = a.per_pair ? p : p / a.k;
            const float v = row_dot<G>(P.w + e * P.expert_bytes, P.chunks, P.K, n, a.img + row * a.img_row_bytes, lane);
            if (lane == 0) P.y[p * P.y_stride + n] = v;
        }
    }
}

template <typename Proj>
int fill(GArgs &a, const uint8_t *img, int64_t row_blocks, int n_proj, const Proj *projs) {
    a.img = img;
    a.img_row_bytes = row_blocks * Q8_1_BYTES;
    a.n_proj = n_proj;
    int strips = 0;
    for (int j = 0; j < n_proj; j++) {
        GProj &p = a.p[j];
        p.w = static_cast<const uint8_t *>(projs[j].w);
        p.y = projs[j].y;
        p.N = (int)projs[j].N;
        p.K = (int)projs[j].K;
        p.y_stride = p.N;
        p.chunks = (int)ceil_div(p.K, UNIT_COLS);
        p.strip_base = strips;
        p.expert_bytes = packed_bytes(projs[j].wtype, p.N, p.K);
        strips += (int)ceil_div(p.N, STRIP_ROWS);
    }
    return strips;
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
    const int strips = fill(a, img, row_blocks, n_proj, projs);
    for (int j = 0; j < n_proj; j++) a.p[j].y_stride = projs[j].y_stride;
    a.T = T;
    a.live = live;
    return launch_pdl("mmvq_g", projs[0].wtype == QK_W_Q4_G64 ? mmvq_g_kernel<64> : mmvq_g_kernel<128>,
                      dim3((unsigned)strips), dim3(256), 0, s, a);
}

qk_status launch_mmvq_g_id(const uint8_t *img, int64_t row_blocks, int rows, int k, int n_proj,
                           const qk_proj_id *projs, const int32_t *counts, const int32_t *offsets,
                           const int32_t *items, bool per_pair, cudaStream_t s) {
    GArgs a = {};
    const int strips = fill(a, img, row_blocks, n_proj, projs);
    a.T = rows;
    a.k = k;
    a.E = projs[0].n_experts;
    a.per_pair = per_pair;
    a.counts = counts;
    a.offsets = offsets;
    a.items = items;
    return launch_pdl("mmvq_g_id", projs[0].wtype == QK_W_Q4_G64 ? mmvq_g_id_kernel<64> : mmvq_g_id_kernel<128>,
                      dim3((unsigned)strips, (unsigned)a.E), dim3(256), 0, s, a);
}

}  // namespace qk

// Routed prefill: matrix products grouped by expert with ragged sizes on a Q8_0 activation image
// (the GEMMs of minfer doc 52 "r49 A-quantize prepass shared-A dedup", section 1, over the grouped
// plan of TensorFold PR #1047 "The fix"; llama.cpp PR #117 Coverage: the image is independent of
// route ids).
//
//   y[p][n] = bf16( sum_i W_e[n][i] * x_row(p)[i] ),  W = (nibble - z) * d_w,  x = q * d_a

#include <cuda_bf16.h>

#include "qk_internal.cuh"

namespace qk {
namespace {

constexpr int MAX_PROJ = 8;
constexpr unsigned FULL = 0xffffffffu;

struct IdProj {
    const uint8_t *w;
    uint16_t *y;
    int64_t y_stride, expert_bytes;
    int N, K, chunks, row_base, wtype;
};
struct IdArgs {
    const int8_t *qs;
    const uint16_t *d;
    int64_t row_blocks;
    const int32_t *counts, *offsets, *items;
    int rows, k, E, per_pair, n_proj;
    IdProj p[MAX_PROJ];
};

// word t of row n's block b, its scale and its zero point
__device__ __forceinline__ uint32_t weight_word(const IdProj &P, const uint8_t *w, int n, int b, int t, float &dw,
                                                int &z) {
    if (P.wtype == QK_W_Q4_0) {
        const uint8_t *unit = w + ((int64_t)(n / UNIT_ROWS) * P.chunks + (b >> 2)) * Q4_UNIT_BYTES;
        const int r = n % UNIT_ROWS, jb = b & 3, g = r & 7, i = (r >> 3) & 3;
        const int grp = r >> 4;
        dw = __half2float(*reinterpret_cast<const __half *>(unit + 8192 + jb * 256 + g * 32 + grp * 4 + 2 * (i & 1)));
        z = 8;
        return *reinterpret_cast<const uint32_t *>(unit + jb * Q4_BLOCK_STRIDE + (r >> 5) * 512 + (4 * g + t) * 16 +
                                                   4 * i);
    }
    const int G = P.wtype == QK_W_Q4_G64 ? 64 : 128, ub = strip_unit_bytes(G);
    const uint8_t *unit = w + ((int64_t)(n / STRIP_ROWS) * P.chunks + (b >> 2)) * ub;
    const int r = n % STRIP_ROWS, jb = b & 3, g = r & 7, i = r >> 3;
    const uint32_t head = *reinterpret_cast<const uint32_t *>(unit + STRIP_DATA + 128 * (jb * QB / G) + 16 * g + 4 * i);
    dw = __half2float(__ushort_as_half((unsigned short)head));
    z = 8 + (int)__half2float(__ushort_as_half((unsigned short)(head >> 16)));
    return *reinterpret_cast<const uint32_t *>(unit + jb * 512 + (4 * g + t) * 16 + 4 * i);
}

// grid (8-row groups of every projection, experts): a warp per row, the expert's pairs one by one.
__global__ void __launch_bounds__(256) mmq_id_kernel(const __grid_constant__ IdArgs a) {
    pdl_trigger();
    pdl_wait();
    int j = 0;
    while (j + 1 < a.n_proj && (int)blockIdx.x >= a.p[j + 1].row_base) j++;
    const IdProj &P = a.p[j];
    const int lane = threadIdx.x & 31, e = blockIdx.y, pairs = a.rows * a.k;
    const int n = ((int)blockIdx.x - P.row_base) * 8 + (threadIdx.x >> 5);
    if (n >= P.N) return;
    const int cnt = min(max(a.counts[e], 0), pairs);
    const int64_t first = a.offsets[e];
    const uint8_t *w = P.w + e * P.expert_bytes;
    for (int c = 0; c < cnt; c++) {
        const int64_t pos = first + c;
        if (pos < 0 || pos >= pairs) continue;
        const int p = a.items[pos];
        if (p < 0 || p >= pairs) continue;
        const int64_t row = a.per_pair ? p : p / a.k;
        float acc = 0.0f;
        for (int b = lane; b < P.K / QB; b += 32) {
            const int8_t *q = a.qs + (row * a.row_blocks + b) * QB;
            int D = 0;
            float dw;
            for (int t = 0; t < 4; t++) {
                int z;
                const uint32_t v = weight_word(P, w, n, b, t, dw, z);
                for (int i = 0; i < 4; i++) {
                    D += ((int)((v >> (8 * i)) & 15) - z) * q[4 * t + i];
                    D += ((int)((v >> (8 * i + 4)) & 15) - z) * q[16 + 4 * t + i];
                }
            }
            acc = fmaf(dw, __half2float(__ushort_as_half(a.d[row * a.row_blocks + b])) * (float)D, acc);
        }
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(FULL, acc, o);
        if (lane == 0) P.y[p * P.y_stride + n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc));
    }
}

}  // namespace

int64_t mmq_id_workspace_bytes(int64_t img_rows, int64_t kmax) { return (img_rows * kmax * 2 + 127) / 128 * 128; }

qk_status launch_mmq_id(const int8_t *qs, const uint16_t *d, int64_t row_blocks, int64_t img_rows, int rows, int k,
                        int n_proj, const qk_proj_id16 *projs, const int32_t *counts, const int32_t *offsets,
                        const int32_t *items, bool per_pair, void *ws, cudaStream_t s) {
    IdArgs a = {};
    a.qs = qs;
    a.d = d;
    a.row_blocks = row_blocks;
    a.counts = counts;
    a.offsets = offsets;
    a.items = items;
    a.rows = rows;
    a.k = k;
    a.E = projs[0].n_experts;
    a.per_pair = per_pair;
    a.n_proj = n_proj;
    int groups = 0;
    for (int j = 0; j < n_proj; j++) {
        IdProj &p = a.p[j];
        p.w = static_cast<const uint8_t *>(projs[j].w);
        p.y = projs[j].y;
        p.y_stride = projs[j].y_stride;
        p.N = (int)projs[j].N;
        p.K = (int)projs[j].K;
        p.chunks = (int)ceil_div(p.K, UNIT_COLS);
        p.wtype = projs[j].wtype;
        p.expert_bytes = packed_bytes(p.wtype, p.N, p.K);
        p.row_base = groups;
        groups += (int)ceil_div(p.N, 8);
    }
    return launch_pdl("mmq_id", mmq_id_kernel, dim3((unsigned)groups, (unsigned)a.E), dim3(256), 0, s, a);
}

}  // namespace qk

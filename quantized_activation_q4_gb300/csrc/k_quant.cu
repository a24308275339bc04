// Q8 activation images and the producers that emit them.
//
//   quantize_q8_1 / quantize_q8_0 : standalone quantisers (llama.cpp PR #117
//       "activation image emission", Coverage: the standard Q8_1 image;
//       minfer doc 52 "r49 A-quantize prepass shared-A dedup", section 1: the
//       Q8_0 prepass with per-32-block amax, rintf scaling and zero pad).
//   rmsnorm_q8_1 / glu_q8_1       : producers that write their original F32
//       output and the Q8_1 image of exactly the stored values (PR #117,
//       Coverage: RMS and F32 GLU producers emit the image).
//
// Work layout: every quant block of 32 elements is handled by 8 consecutive
// lanes, 4 elements each, so a warp quantises 4 blocks at once with 3-step
// xor shuffles for the block max and the code sum. All block arithmetic is
// binary32 with IEEE division (no fast-math in this file), the codes use
// round-to-nearest-even and the halves use __float2half_rn.

#include <cfloat>

#include "qk_internal.cuh"

namespace qk {
namespace {

constexpr unsigned FULL = 0xffffffffu;

// Four consecutive floats from p (16-byte aligned fast path, else scalar with
// a bound: elements at index >= n read as 0).
__device__ __forceinline__ void load4(const float *p, int n, float v[4]) {
    if (n >= 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const float4 t = ld_prev(reinterpret_cast<const float4 *>(p));
        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = i < n ? ld_prev(p + i) : 0.0f;
    }
}

__device__ __forceinline__ void store4(float *p, const float v[4]) {
    if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) p[i] = v[i];
    }
}

// Quantises one 32-element block held by 8 lanes (4 values each; j8 = the
// lane's index in its group). All 32 lanes of the warp must call this.
// Returns the binary32 scale d; codes are packed little-endian into *codes
// and the block's code sum into *sum.
// ZEROS: for inputs where exact zeros are common (ReGLU outputs: half of them), zeros skip the
// division (the same codes; a division of zero measured slower on this GPU).
template <bool ZEROS = false>
__device__ __forceinline__ float q8_block(const float v[4], uint32_t *codes, int *sum) {
    float a = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
    a = fmaxf(a, __shfl_xor_sync(FULL, a, 1));
    a = fmaxf(a, __shfl_xor_sync(FULL, a, 2));
    a = fmaxf(a, __shfl_xor_sync(FULL, a, 4));
    const float d = a / 127.0f;
    int q[4] = {0, 0, 0, 0};
    if (a != 0.0f) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (ZEROS) {   // a zero's code is 0: its quotient is taken as 1 / 1 and dropped
                const bool z = v[i] == 0.0f;
                const int qi = __float2int_rn((z ? d : v[i]) / d);
                q[i] = z ? 0 : qi;
            } else {
                q[i] = __float2int_rn(v[i] / d);
            }
        }
    }
    int s = q[0] + q[1] + q[2] + q[3];
    s += __shfl_xor_sync(FULL, s, 1);
    s += __shfl_xor_sync(FULL, s, 2);
    s += __shfl_xor_sync(FULL, s, 4);
    *codes = (uint32_t)(q[0] & 0xff) | ((uint32_t)(q[1] & 0xff) << 8) |
             ((uint32_t)(q[2] & 0xff) << 16) | ((uint32_t)(q[3] & 0xff) << 24);
    *sum = s;
    return d;
}

// Writes lane j8's share of a Q8_1 block: codes at bytes 4+4*j8, and for
// j8 == 0 the header [half d][half d*sum].
__device__ __forceinline__ void put_q8_1(uint8_t *blk, int j8, float d, uint32_t codes, int sum) {
    reinterpret_cast<uint32_t *>(blk + 4)[j8] = codes;
    if (j8 == 0) {
        __half2 h = __halves2half2(__float2half_rn(d), __float2half_rn(d * (float)sum));
        *reinterpret_cast<__half2 *>(blk) = h;
    }
}

// ---------------------------------------------------------------- quantizers
// grid (T, ceil(row_blocks / (G*QPB))), NT threads, G = NT / 8 lane groups: lane group m of
// warp w handles blocks G*QPB*blockIdx.y + G*j + 4*w + m (j < QPB) of row blockIdx.x (rows on
// x: up to 2^31-1). A lane loads its QPB float4s before it quantises, so that large images
// keep several loads per thread in flight, while small ones spread over more CTAs (QPB = 1).
// Large images with rows of at most 128 blocks take a 128-thread CTA per row with QPB =
// ceil(row_blocks / 16) (more rows in flight per SM, few idle lanes), wider rows 256 threads
// with QPB = 4. Every block is quantised on its own, so the bytes do not depend on the shape.
template <bool Q81, int QPB, int NT = 256>
__global__ void __launch_bounds__(NT) quantize_kernel(const float *x, int K,
                                                       int64_t x_stride, uint8_t *__restrict__ out,
                                                       int8_t *__restrict__ qs, uint16_t *__restrict__ dh,
                                                       int64_t row_blocks, int T, const int32_t *live) {
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x;
    const int lane = threadIdx.x & 31, j8 = lane & 7;
    constexpr int G = NT / 8;
    const int64_t b0 = (int64_t)blockIdx.y * G * QPB + (threadIdx.x >> 5) * 4 + (lane >> 3);
    float v[QPB][4];
    // the row's values are loaded together with the live count (row t < T is in the caller's
    // buffer even when it is padding), so the global reads overlap
#pragma unroll
    for (int j = 0; j < QPB; j++) {
        const int64_t b = b0 + G * j, col = b * QB + 4 * j8;
        v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.0f;
        if (b < row_blocks && col < K) load4(x + t * x_stride + col, (int)(K - col < 4 ? K - col : 4), v[j]);
    }
    if (t >= live_rows(live, T)) return;
#pragma unroll
    for (int j = 0; j < QPB; j++) {
        const int64_t b = b0 + G * j;
        uint32_t codes;
        int sum;
        const float d = q8_block(v[j], &codes, &sum);   // all lanes take part in the shuffles
        if (b >= row_blocks) continue;                   // whole 8-lane group agrees
        if (Q81) {
            put_q8_1(out + (t * row_blocks + b) * Q8_1_BYTES, j8, d, codes, sum);
        } else {
            reinterpret_cast<uint32_t *>(qs + (t * row_blocks + b) * QB)[j8] = codes;
            if (j8 == 0) dh[t * row_blocks + b] = __half_as_ushort(__float2half_rn(d));
        }
    }
}

// ---------------------------------------------------------------- RMS producer
// One CTA per row; the row stays in registers between the sum of squares and
// the output. The reference shape is 1024 threads (thread i holds columns
// 4i + 4096*it for it < ITEMS, ITEMS = 1, 2, 4 or 8 by K, so K <= 32768). For
// many rows a smaller CTA takes the row instead (128 threads for K <= 4096,
// eight rows in flight per SM; 256 threads for K <= 8192, four): its thread j
// plays the reference threads j + NT*m (m < 1024 / NT) and reduces their
// partial sums in the same order (one warp tree per m, then the same 32-entry
// tree), so the bits are those of the 1024-thread shape.
// With ITEMS <= 2 the weight and bias are loaded together with the row, before
// the reduction.
constexpr int RMS_THREADS = 1024;
constexpr int RMS_ITEMS = 8;
constexpr int RMS_ROWS_FOR_SMALL = 256;   // rows from which the 256-thread shape is used

// Q81: the image is Q8_1 blocks (img); else Q8_0 split planes (qs codes, dh half scales), the
// prefill layout that qk_mmq reads.
template <int NT, int ITEMS, bool Q81>
__global__ void __launch_bounds__(NT, RMS_THREADS / NT) rmsnorm_q8_1_kernel(
    const float *x, int K, int64_t x_stride, int kind, const float *w,
    const float *bias, float scale, float eps, float *__restrict__ y, int64_t y_stride,
    uint8_t *__restrict__ img, int8_t *__restrict__ qs, uint16_t *__restrict__ dh, int64_t row_blocks, int T,
    const int32_t *live) {
    constexpr bool EARLY = ITEMS <= 2;   // registers for the weight and bias next to the row
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x;
    const float *xr = x + t * x_stride;
    const int tid = threadIdx.x, lane = tid & 31, j8 = lane & 7;
    const bool use_w = kind == QK_NORM_MUL || kind == QK_NORM_MUL_ADD, use_b = kind == QK_NORM_MUL_ADD;

    // the row (and with EARLY its weight and bias) is loaded together with the live count (row
    // t < T is in the caller's buffer even when it is padding), so the global reads overlap
    float v[ITEMS][4], wv[EARLY ? ITEMS : 1][4], bv[EARLY ? ITEMS : 1][4];
#pragma unroll
    for (int it = 0; it < ITEMS; it++) {
        const int c = 4 * tid + 4 * NT * it;
        v[it][0] = v[it][1] = v[it][2] = v[it][3] = 0.0f;
        if (c < K) {
            load4(xr + c, 4, v[it]);
            if (EARLY && use_w) load4(w + c, 4, wv[EARLY ? it : 0]);
            if (EARLY && use_b) load4(bias + c, 4, bv[EARLY ? it : 0]);
        }
    }
    if (t >= live_rows(live, T)) return;
    // reference thread j + NT*m holds items m, m + R, m + 2R, ... of this thread (R = 1024 / NT)
    constexpr int R = RMS_THREADS / NT;
    __shared__ float red[RMS_THREADS / 32];
#pragma unroll
    for (int m = 0; m < R; m++) {
        float ss = 0.0f;
#pragma unroll
        for (int it = m; it < ITEMS; it += R)
            ss += v[it][0] * v[it][0] + v[it][1] * v[it][1] + v[it][2] * v[it][2] + v[it][3] * v[it][3];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
        if (lane == 0) red[(tid >> 5) + m * (NT / 32)] = ss;
    }
    __syncthreads();
    if (tid < 32) {
        float tot = red[tid];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(FULL, tot, o);
        if (tid == 0) red[0] = 1.0f / sqrtf(tot / (float)K + eps);
    }
    __syncthreads();
    const float r = red[0];

    float *yr = y + t * y_stride;
    uint8_t *ir = Q81 ? img + t * row_blocks * Q8_1_BYTES : nullptr;
    int8_t *qr = Q81 ? nullptr : qs + t * row_blocks * QB;
    uint16_t *dr = Q81 ? nullptr : dh + t * row_blocks;
#pragma unroll
    for (int it = 0; it < ITEMS; it++) {
        if (4 * NT * it >= K) break;                        // uniform: no warp has columns left
        const int c = 4 * tid + 4 * NT * it;
        const bool ok = c < K;                               // K % 32 == 0: whole 8-lane groups agree
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        if (ok) {
            float wl[4], bl[4];
            const float *wq = wl, *bq = bl;
            if (EARLY) {
                wq = wv[EARLY ? it : 0];
                bq = bv[EARLY ? it : 0];
            } else {
                if (use_w) load4(w + c, 4, wl);
                if (use_b) load4(bias + c, 4, bl);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                float q = v[it][i] * r;
                if (kind == QK_NORM_MUL) q = q * wq[i];
                else if (kind == QK_NORM_MUL_ADD) q = q * wq[i] + bq[i];
                else if (kind == QK_NORM_SCALE) q = q * scale;
                o[i] = q;
            }
            store4(yr + c, o);
        }
        uint32_t codes;
        int sum;
        const float d = q8_block(o, &codes, &sum);   // all lanes of the warp take part
        if (ok) {
            if (Q81) {
                put_q8_1(ir + (int64_t)(c / QB) * Q8_1_BYTES, j8, d, codes, sum);
            } else {
                reinterpret_cast<uint32_t *>(qr + (int64_t)(c / QB) * QB)[j8] = codes;
                if (j8 == 0) dr[c / QB] = __half_as_ushort(__float2half_rn(d));
            }
        }
    }
    // zero blocks of the row padding
    for (int64_t bb = K / QB + tid; bb < row_blocks; bb += NT) {
        if (Q81) {
            uint32_t *p = reinterpret_cast<uint32_t *>(ir + bb * Q8_1_BYTES);
#pragma unroll
            for (int i = 0; i < 9; i++) p[i] = 0u;
        } else {
            uint32_t *p = reinterpret_cast<uint32_t *>(qr + bb * QB);
#pragma unroll
            for (int i = 0; i < 8; i++) p[i] = 0u;
            dr[bb] = 0;
        }
    }
}

// ---------------------------------------------------------------- GLU producer
// act(g) * u for the GLU kinds; SwiGLU-OAI and SwiGLU-clamp clamp g from above and u both
// ways at limit (SwiGLU-OAI also scales the gate by alpha and multiplies by u + 1).
__device__ __forceinline__ float glu_out(int kind, float g, float u, float alpha, float limit) {
    switch (kind) {
        case QK_GLU_SWIGLU: return g / (1.0f + expf(-g)) * u;
        case QK_GLU_GEGLU_TANH: {
            const float c = 0.7978845608028654f;  // sqrt(2/pi)
            return 0.5f * g * (1.0f + tanhf(c * (g + 0.044715f * g * g * g))) * u;
        }
        case QK_GLU_GEGLU_ERF: return 0.5f * g * (1.0f + erff(g * 0.7071067811865476f)) * u;
        case QK_GLU_GEGLU_QUICK: return g / (1.0f + expf(-1.702f * g)) * u;
        case QK_GLU_SWIGLU_OAI: {
            const float x = fminf(g, limit), v = fminf(fmaxf(u, -limit), limit);
            return x / (1.0f + expf(-alpha * x)) * (v + 1.0f);
        }
        case QK_GLU_SWIGLU_CLAMP: {
            const float x = fminf(g, limit), v = fminf(fmaxf(u, -limit), limit);
            return x / (1.0f + expf(-x)) * v;
        }
        default: return fmaxf(g, 0.0f) * u;
    }
}

// grid (T, ceil(N/1024)), 256 threads; thread i of CTA (t, cy) handles columns 1024*cy + 4i of row t.
__global__ void __launch_bounds__(256) glu_q8_1_kernel(
    int kind, int layout, const float *a, int64_t a_stride, const float *b,
    int64_t b_stride, int N, float *__restrict__ out, int64_t out_stride, uint8_t *__restrict__ img,
    int64_t row_blocks, int T, float alpha, float limit, const int32_t *live) {
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x;
    const int tid = threadIdx.x, j8 = tid & 7;
    const int c = blockIdx.y * 1024 + 4 * tid;
    const float *g, *u;
    if (layout == QK_GLU_SEPARATE) {
        g = a + t * a_stride;
        u = b + t * b_stride;
    } else if (layout == QK_GLU_PACKED) {
        g = a + t * a_stride;
        u = g + N;
    } else {
        u = a + t * a_stride;
        g = u + N;
    }
    const bool ok = c < N;
    // the inputs are loaded together with the live count (row t < T is in the caller's
    // buffers even when it is padding), so the global reads overlap
    float gv[4] = {0.f, 0.f, 0.f, 0.f}, uv[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok) {
        load4(g + c, 4, gv);
        load4(u + c, 4, uv);
    }
    if (t >= live_rows(live, T)) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok) {
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = glu_out(kind, gv[i], uv[i], alpha, limit);
        store4(out + t * out_stride + c, v);
    }
    uint32_t codes;
    int sum;
    const float d = kind == QK_GLU_REGLU ? q8_block<true>(v, &codes, &sum) : q8_block(v, &codes, &sum);
    uint8_t *ir = img + t * row_blocks * Q8_1_BYTES;
    if (ok) put_q8_1(ir + (int64_t)(c / QB) * Q8_1_BYTES, j8, d, codes, sum);
    if (blockIdx.y == 0) {  // zero blocks of the row padding
        for (int64_t bb = N / QB + tid; bb < row_blocks; bb += 256) {
            uint32_t *p = reinterpret_cast<uint32_t *>(ir + bb * Q8_1_BYTES);
#pragma unroll
            for (int i = 0; i < 9; i++) p[i] = 0u;
        }
    }
}

// ---------------------------------------------------------------- GLU producer of the prefill planes
// Input rows of binary32 or bfloat16, codes and half scales as qk_quantize_q8_0 of the binary32 products,
// which are stored only when `out` is given.
//
// Bound by issue slots and, once those are few, by memory. 26600 x 768 bfloat16 pairs (103 MB, 15.3 us at
// the copy rate): with IEEE divisions and expf 90 instructions an element, 59 us; with approximate functions
// 37, 27 us; with two elements to an instruction 29, 23 us (issue 78%). 700 x 18944 binary32 pairs with
// their products stored (161 MB, 23.8 us): 36, 27.4 and 24.5 us. One, three or four blocks a thread and
// other numbers of CTAs per SM change less than 2%.
//   - the sigmoid kinds are g / (1 + 2^(-c g)) with ex2.approx and rcp.approx, two elements to an
//     instruction elsewhere. Relative errors: the exponent's rounding |c g| 2^-24 and 2^-22 of ex2, weighted
//     by the sigmoid's share e / (1 + e), and 2^-23 each of rcp and the products: below 1e-6 of the result or
//     3e-7 of |g u| everywhere. GeGLU-tanh is one of them: 0.5 (1 + tanh z) = 1 / (1 + e^(-2z)), with no
//     cancellation;
//   - d = m / 127 by a product and one correction step (Brisebarre, Muller, Raina, "Accelerating correctly
//     rounded floating-point division when the divisor is known in advance"): the same as a division for
//     every significand where nothing under- or overflows;
//   - codes are rint(x * r), r the approximate reciprocal of d. x r is off x / d by at most 127 (2^-23 + 2^-24
//     + 2^-24) = 3.1e-5 and so gives another code only that near to a tie: blocks with an element within
//     4e-5 of one (and scales outside 1e-30 .. 1e30) divide, so the bytes are qk_quantize_q8_0's.
// A group of four lanes has a quant block, eight columns a lane; a thread has two blocks' loads in flight.
// A CTA of 64 groups takes 128 consecutive blocks of a row, or as many whole rows as 128 blocks hold.

// Two binary32 values in a register pair, and operations on both.
typedef uint64_t F2;
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo(F2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi(F2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 both(float v) { return f2(v, v); }
// max(|m|, |v|, |w|): NaN is left out, or (NAN_TOO) the result
template <bool NAN_TOO>
__device__ __forceinline__ float max3(float m, F2 v) {
    float r;
    if (NAN_TOO)
        asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(lo(v)), "f"(hi(v)));
    else
        asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(lo(v)), "f"(hi(v)));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// x / (1 + e^-y), c = -log2(e) y
__device__ __forceinline__ F2 gated(F2 x, F2 c) {
    const F2 s = add2(f2(ex2(lo(c)), ex2(hi(c))), both(1.0f));
    return mul2(x, f2(rcp(lo(s)), rcp(hi(s))));
}
constexpr float LOG2E = 1.4426950408889634f;

template <int KIND>
__device__ __forceinline__ F2 glu_pair(F2 g, F2 u, float alpha_log2e, float limit) {
    if (KIND == QK_GLU_SWIGLU) return mul2(gated(g, mul2(g, both(-LOG2E))), u);
    if (KIND == QK_GLU_GEGLU_TANH) {   // 2 sqrt(2/pi) log2(e) (g + 0.044715 g^3)
        const F2 t = fma2(mul2(g, both(0.044715f)), g, both(1.0f));
        return mul2(gated(g, mul2(mul2(g, both(-2.0f * 0.7978845608028654f * LOG2E)), t)), u);
    }
    if (KIND == QK_GLU_GEGLU_QUICK) return mul2(gated(g, mul2(g, both(-1.702f * LOG2E))), u);
    if (KIND == QK_GLU_SWIGLU_OAI || KIND == QK_GLU_SWIGLU_CLAMP) {
        const F2 x = f2(fminf(lo(g), limit), fminf(hi(g), limit));
        const F2 v = f2(fminf(fmaxf(lo(u), -limit), limit), fminf(fmaxf(hi(u), -limit), limit));
        return KIND == QK_GLU_SWIGLU_OAI ? mul2(gated(x, mul2(x, both(-alpha_log2e))), add2(v, both(1.0f)))
                                         : mul2(gated(x, mul2(x, both(-LOG2E))), v);
    }
    return f2(glu_out(KIND, lo(g), lo(u), 0.0f, 0.0f), glu_out(KIND, hi(g), hi(u), 0.0f, 0.0f));   // GeGLU-erf, ReGLU
}

// Eight columns as they are in memory: loads in flight cost few registers.
template <bool BF16>
struct Raw8 {
    uint4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *p, int64_t i, bool wide) {
        const uint8_t *q = static_cast<const uint8_t *>(p) + i * (BF16 ? 2 : 4);
        if (wide) {
#pragma unroll
            for (int h = 0; h < (BF16 ? 1 : 2); h++) w[h] = ld_prev(reinterpret_cast<const uint4 *>(q) + h);
        } else {
            uint32_t x[BF16 ? 4 : 8];
#pragma unroll
            for (int j = 0; j < (BF16 ? 4 : 8); j++) {
                if (BF16)
                    x[j] = ld_prev(reinterpret_cast<const uint16_t *>(q) + 2 * j) |
                           (uint32_t)ld_prev(reinterpret_cast<const uint16_t *>(q) + 2 * j + 1) << 16;
                else
                    x[j] = ld_prev(reinterpret_cast<const uint32_t *>(q) + j);
            }
#pragma unroll
            for (int h = 0; h < (BF16 ? 1 : 2); h++) w[h] = make_uint4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
        }
    }
    __device__ __forceinline__ F2 pair(int i) const {   // columns 2i, 2i + 1
        const uint4 v = w[BF16 ? 0 : i >> 1];
        if (BF16) {
            const uint32_t x = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
            return f2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
        }
        return i & 1 ? f2(__uint_as_float(v.z), __uint_as_float(v.w)) : f2(__uint_as_float(v.x), __uint_as_float(v.y));
    }
};

// wide: every eight columns of a and b are 16-byte aligned. Groups over whole rows (rows_per_cta > 1):
// row_mul = ceil(2^16 / blocks of a row), exact for the quotients of 0..63 here.
template <int KIND, bool BF16>
__global__ void __launch_bounds__(256, BF16 ? 6 : 4) glu_q8_0_kernel(
    int layout, bool wide, const void *a, int64_t a_stride, const void *b, int64_t b_stride,
    int N, float *__restrict__ out, int64_t out_stride, int8_t *__restrict__ qs, uint16_t *__restrict__ dh,
    int64_t row_blocks, int T, int rows_per_cta, uint32_t row_mul, int step_row, int step_blk, float alpha, float limit,
    const int32_t *live) {
    pdl_trigger();
    pdl_wait();
    const int kb = N / QB, group = threadIdx.x >> 2, l4 = threadIdx.x & 3;
    int64_t row[2];
    int blk[2];
    Raw8<BF16> g[2], u[2];
    int r0 = 0;
    blk[0] = blockIdx.y * 128 + group;
    if (rows_per_cta > 1) {   // the second block is 64 groups on
        r0 = (group * row_mul) >> 16;
        blk[0] = group - r0 * kb;
    }
    bool on[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        if (h == 1) {
            blk[1] = blk[0] + step_blk;
            r0 += step_row;
            if (rows_per_cta > 1 && blk[1] >= kb) {
                blk[1] -= kb;
                r0++;
            }
        }
        row[h] = (int64_t)blockIdx.x * rows_per_cta + r0;
        on[h] = r0 < rows_per_cta && row[h] < T && blk[h] < kb;
        // loaded together with the live count (row < T is in the caller's buffers even when it is padding);
        // a group without a block loads the first one's columns again
        const int64_t r = on[h] ? row[h] : 0, c = (on[h] ? blk[h] : 0) * QB + 8 * l4, first = r * a_stride + c;
        g[h].load(a, layout == QK_GLU_PACKED_SWAPPED ? first + N : first, wide);
        if (layout == QK_GLU_SEPARATE)
            u[h].load(b, r * b_stride + c, wide);
        else
            u[h].load(a, layout == QK_GLU_PACKED ? first + N : first, wide);
    }
    const int n_live = live_rows(live, T);
    const float alpha_log2e = fminf(fmaxf(alpha * LOG2E, -FLT_MAX), FLT_MAX);   // finite: a gate of zero stays zero
#pragma unroll
    for (int h = 0; h < 2; h++) {
        F2 v[4];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = glu_pair<KIND>(g[h].pair(i), u[h].pair(i), alpha_log2e, limit);
            m = max3<false>(m, v[i]);
        }
        m = fmaxf(m, __shfl_xor_sync(FULL, m, 1));
        m = fmaxf(m, __shfl_xor_sync(FULL, m, 2));
        if (!on[h] || row[h] >= n_live) continue;   // a block's four lanes agree
        constexpr float C = 1.0f / 127.0f;
        float d = m * C;
        d = fmaf(fmaf(-127.0f, d, m), C, d);
        const F2 inv = both(rcp(d));
        constexpr float MAGIC = 12582912.0f;   // 1.5 * 2^23: the sum's low byte is the rounded code
        uint32_t t[8];
        float off = 0.0f;   // the farthest from a code
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const F2 r = mul2(v[i], inv), s = add2(r, both(MAGIC));
            t[2 * i] = __float_as_uint(lo(s));
            t[2 * i + 1] = __float_as_uint(hi(s));
            off = max3<true>(off, fma2(add2(s, both(-MAGIC)), both(-1.0f), r));
        }
        if (!(d > 1e-30f && d < 1e30f && off < 0.5f - 4.0e-5f)) {   // also with a NaN anywhere
            d = m / 127.0f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                t[2 * i] = m != 0.0f ? (uint32_t)__float2int_rn(lo(v[i]) / d) : 0u;
                t[2 * i + 1] = m != 0.0f ? (uint32_t)__float2int_rn(hi(v[i]) / d) : 0u;
            }
        }
        const uint32_t c0 = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
        const uint32_t c1 = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
        if (out) {
            float *o = out + row[h] * out_stride + blk[h] * QB + 8 * l4;
            const float w[8] = {lo(v[0]), hi(v[0]), lo(v[1]), hi(v[1]), lo(v[2]), hi(v[2]), lo(v[3]), hi(v[3])};
            store4(o, w);
            store4(o + 4, w + 4);
        }
        const int64_t at = row[h] * row_blocks + blk[h];
        uint32_t *q = reinterpret_cast<uint32_t *>(qs + at * QB) + 2 * l4;
        if ((reinterpret_cast<uintptr_t>(q) & 7u) == 0) {
            *reinterpret_cast<uint2 *>(q) = make_uint2(c0, c1);
        } else {
            q[0] = c0;
            q[1] = c1;
        }
        if (l4 == 0) dh[at] = __half_as_ushort(__float2half_rn(d));
    }
    if (blockIdx.y == 0 && kb < row_blocks) {   // zero blocks of the rows' padding
        for (int r = 0; r < rows_per_cta; r++) {
            const int64_t t = (int64_t)blockIdx.x * rows_per_cta + r;
            if (t >= n_live) break;
            for (int64_t bb = kb + threadIdx.x; bb < row_blocks; bb += 256) {
                uint32_t *p = reinterpret_cast<uint32_t *>(qs + (t * row_blocks + bb) * QB);
#pragma unroll
                for (int i = 0; i < 8; i++) p[i] = 0u;
                dh[t * row_blocks + bb] = 0;
            }
        }
    }
}

constexpr int64_t QUANT_BIG_BLOCKS = 1 << 17;   // blocks per call from which QPB = 4 is used

}  // namespace

// Large images with rows of at most 128 blocks: one 128-thread CTA per row (QPB = ceil(rb / 16)).
template <bool Q81>
static qk_status launch_quantize_rows128(const char *name, const float *x, int T, int K, int64_t x_stride,
                                         uint8_t *img, int8_t *qs, uint16_t *d, int64_t row_blocks,
                                         const int32_t *live, cudaStream_t s) {
    const int qpb = (int)ceil_div(row_blocks, 16);
    auto kernel = qpb <= 5   ? quantize_kernel<Q81, 5, 128>
                  : qpb == 6 ? quantize_kernel<Q81, 6, 128>
                  : qpb == 7 ? quantize_kernel<Q81, 7, 128>
                             : quantize_kernel<Q81, 8, 128>;
    return launch_pdl(name, kernel, dim3((unsigned)T, 1u), dim3(128), 0, s, x, K, x_stride, img, qs, d, row_blocks,
                      T, live);
}

qk_status launch_quantize_q8_1(const float *x, int T, int K, int64_t x_stride, uint8_t *img,
                               int64_t row_blocks, const int32_t *live, cudaStream_t s) {
    if (T == 0) return QK_OK;
    const bool big = (int64_t)T * row_blocks >= QUANT_BIG_BLOCKS;
    if (big && row_blocks > 64 && row_blocks <= 128)
        return launch_quantize_rows128<true>("quantize_q8_1", x, T, K, x_stride, img, nullptr, nullptr, row_blocks,
                                             live, s);
    dim3 grid((unsigned)T, (unsigned)ceil_div(row_blocks, big ? 128 : 32));
    return launch_pdl("quantize_q8_1", big ? quantize_kernel<true, 4> : quantize_kernel<true, 1>, grid, dim3(256),
                      0, s, x, K, x_stride, img, (int8_t *)nullptr, (uint16_t *)nullptr, row_blocks, T, live);
}

qk_status launch_quantize_q8_0(const float *x, int T, int K, int64_t x_stride, int8_t *qs,
                               uint16_t *d, int64_t row_blocks, const int32_t *live, cudaStream_t s) {
    if (T == 0) return QK_OK;
    const bool big = (int64_t)T * row_blocks >= QUANT_BIG_BLOCKS;
    if (big && row_blocks > 64 && row_blocks <= 128)
        return launch_quantize_rows128<false>("quantize_q8_0", x, T, K, x_stride, nullptr, qs, d, row_blocks, live,
                                              s);
    dim3 grid((unsigned)T, (unsigned)ceil_div(row_blocks, big ? 128 : 32));
    return launch_pdl("quantize_q8_0", big ? quantize_kernel<false, 4> : quantize_kernel<false, 1>, grid,
                      dim3(256), 0, s, x, K, x_stride, (uint8_t *)nullptr, qs, d, row_blocks, T, live);
}

template <bool Q81>
static qk_status launch_rmsnorm(const float *x, int T, int K, int64_t x_stride, int kind, const float *w,
                                const float *b, float scale, float eps, float *y, int64_t y_stride, uint8_t *img,
                                int8_t *qs, uint16_t *dh, int64_t row_blocks, const int32_t *live, cudaStream_t s) {
    if (T == 0) return QK_OK;
    const int per = 4 * RMS_THREADS;   // columns per item of the reference shape
    if (T >= RMS_ROWS_FOR_SMALL && K <= 2 * per) {   // 256 threads, four times the items
        if (K <= per)   // 128 threads: eight rows in flight per SM
            return launch_pdl(Q81 ? "rmsnorm_q8_1" : "rmsnorm_q8_0", rmsnorm_q8_1_kernel<128, 8, Q81>,
                              dim3((unsigned)T), dim3(128), 0, s, x, K, x_stride, kind, w, b, scale, eps, y, y_stride,
                              img, qs, dh, row_blocks, T, live);
        return launch_pdl(Q81 ? "rmsnorm_q8_1" : "rmsnorm_q8_0", rmsnorm_q8_1_kernel<256, 8, Q81>, dim3((unsigned)T),
                          dim3(256), 0, s, x, K, x_stride, kind, w, b, scale, eps, y, y_stride, img, qs, dh,
                          row_blocks, T, live);
    }
    auto kernel = K <= per ? rmsnorm_q8_1_kernel<RMS_THREADS, 1, Q81>
                  : K <= 2 * per ? rmsnorm_q8_1_kernel<RMS_THREADS, 2, Q81>
                  : K <= 4 * per ? rmsnorm_q8_1_kernel<RMS_THREADS, 4, Q81>
                                 : rmsnorm_q8_1_kernel<RMS_THREADS, RMS_ITEMS, Q81>;
    return launch_pdl(Q81 ? "rmsnorm_q8_1" : "rmsnorm_q8_0", kernel, dim3((unsigned)T), dim3(RMS_THREADS), 0, s, x,
                      K, x_stride, kind, w, b, scale, eps, y, y_stride, img, qs, dh, row_blocks, T, live);
}

qk_status launch_rmsnorm_q8_1(const float *x, int T, int K, int64_t x_stride, int kind,
                              const float *w, const float *b, float scale, float eps, float *y,
                              int64_t y_stride, uint8_t *img, int64_t row_blocks,
                              const int32_t *live, cudaStream_t s) {
    return launch_rmsnorm<true>(x, T, K, x_stride, kind, w, b, scale, eps, y, y_stride, img, nullptr, nullptr,
                                row_blocks, live, s);
}

qk_status launch_rmsnorm_q8_0(const float *x, int T, int K, int64_t x_stride, int kind, const float *w,
                              const float *b, float scale, float eps, float *y, int64_t y_stride, int8_t *qs,
                              uint16_t *dh, int64_t row_blocks, const int32_t *live, cudaStream_t s) {
    return launch_rmsnorm<false>(x, T, K, x_stride, kind, w, b, scale, eps, y, y_stride, nullptr, qs, dh,
                                 row_blocks, live, s);
}

qk_status launch_glu_q8_1(int kind, int layout, const float *a, int64_t a_stride, const float *b,
                          int64_t b_stride, int T, int N, float *out, int64_t out_stride,
                          uint8_t *img, int64_t row_blocks, float alpha, float limit, const int32_t *live,
                          cudaStream_t s) {
    if (T == 0) return QK_OK;
    dim3 grid((unsigned)T, (unsigned)ceil_div(N, 1024));
    return launch_pdl("glu_q8_1", glu_q8_1_kernel, grid, dim3(256), 0, s, kind, layout, a, a_stride, b, b_stride,
                      N, out, out_stride, img, row_blocks, T, alpha, limit, live);
}

template <bool BF16>
static auto glu_q8_0_of(int kind) -> decltype(&glu_q8_0_kernel<0, BF16>) {
    switch (kind) {
        case QK_GLU_SWIGLU: return glu_q8_0_kernel<QK_GLU_SWIGLU, BF16>;
        case QK_GLU_GEGLU_TANH: return glu_q8_0_kernel<QK_GLU_GEGLU_TANH, BF16>;
        case QK_GLU_REGLU: return glu_q8_0_kernel<QK_GLU_REGLU, BF16>;
        case QK_GLU_GEGLU_ERF: return glu_q8_0_kernel<QK_GLU_GEGLU_ERF, BF16>;
        case QK_GLU_GEGLU_QUICK: return glu_q8_0_kernel<QK_GLU_GEGLU_QUICK, BF16>;
        case QK_GLU_SWIGLU_OAI: return glu_q8_0_kernel<QK_GLU_SWIGLU_OAI, BF16>;
        default: return glu_q8_0_kernel<QK_GLU_SWIGLU_CLAMP, BF16>;
    }
}

qk_status launch_glu_q8_0(int kind, int layout, int elem, const void *a, int64_t a_stride, const void *b,
                          int64_t b_stride, int T, int N, float *out, int64_t out_stride, int8_t *qs, uint16_t *d,
                          int64_t row_blocks, float alpha, float limit, const int32_t *live, cudaStream_t s) {
    if (T == 0) return QK_OK;
    const int kb = N / QB, rows = kb >= 128 ? 1 : 128 / kb;   // rows of a CTA
    const int64_t es = elem == QK_ELEM_BF16 ? 2 : 4;
    const bool separate = layout == QK_GLU_SEPARATE;
    const bool wide = ((reinterpret_cast<uintptr_t>(a) | (uintptr_t)(a_stride * es) |   // N * es is a multiple of 64
                        (separate ? reinterpret_cast<uintptr_t>(b) | (uintptr_t)(b_stride * es) : 0)) &
                       15u) == 0;
    dim3 grid((unsigned)ceil_div(T, rows), (unsigned)(rows > 1 ? 1 : ceil_div(kb, 128)));
    return launch_pdl("glu_q8_0", elem == QK_ELEM_BF16 ? glu_q8_0_of<true>(kind) : glu_q8_0_of<false>(kind), grid,
                      dim3(256), 0, s, layout, wide, a, a_stride, b, b_stride, N, out, out_stride, qs, d, row_blocks, T,
                      rows, (uint32_t)((65536 + kb - 1) / kb), rows > 1 ? 64 / kb : 0, rows > 1 ? 64 % kb : 64, alpha,
                      limit, live);
}

}  // namespace qk

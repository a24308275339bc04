// Tensor-core building blocks shared by the prefill kernels: mbarrier waits with a limit, TMA copies,
// tcgen05 issue, and the conversion of packed nibbles to binary16 A operands.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "qk_internal.cuh"

namespace qk {

constexpr uint32_t SPIN_LIMIT = 1u << 16;
constexpr uint32_t SUSPEND_NS = 20000;

static __device__ unsigned int g_tc_faults = 0;   // one per translation unit; bits as qk_device_faults

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t a, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(a), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t a) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t a, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(a), "r"(bytes) : "memory");
}
// Bounded wait: suspends until the phase completes (or SUSPEND_NS), gives up
// after SPIN_LIMIT tries (about a second at most), records a fault and
// returns false.
__device__ __forceinline__ bool mbar_wait(uint32_t a, uint32_t parity) {
    for (uint32_t i = 0; i < SPIN_LIMIT; i++) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(a), "r"(parity), "r"(SUSPEND_NS)
            : "memory");
        if (ok) return true;
    }
    atomicOr(&g_tc_faults, 1u);
    return false;
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void *src, uint32_t bytes, uint32_t mbar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(mbar)
                 : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar)
        : "memory");
}
// shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 B apart
__device__ __forceinline__ uint64_t sdesc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// instruction descriptor: f32 accumulator, f16 A and B, both K-major, M = 128, N columns (a multiple
// of 16 up to 256)
__host__ __device__ constexpr uint32_t mma_idesc(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// D (tensor memory) (+)= A (tensor memory) x B (shared memory)
__device__ __forceinline__ void tc_mma(uint32_t tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t mbar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(mbar)
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Four weight bytes (word t of one row of a Q4_0 block) -> 16 bytes of f16
// A values (nibble - 8) * dw, K order: e(4t), e(4t+2), e(4t+1), e(4t+3),
// e(16+4t), e(16+4t+2), e(16+4t+1), e(16+4t+3). The nibble becomes an exact
// half by OR-ing it under an exponent (1024 + lo, 64 + hi); subtracting
// 1024 + z / 64 + z leaves the exact nibble - z; one rounding in the multiply by dw.
__device__ __forceinline__ uint32_t a_pair(uint32_t v, __half2 bias, __half2 dw) {
    const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&v), bias), dw);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint4 a_word(uint32_t w, __half2 dw, __half2 blo, __half2 bhi) {
    const uint32_t w8 = w >> 8;
    return make_uint4(a_pair((w & 0x000F000Fu) | 0x64006400u, blo, dw), a_pair((w8 & 0x000F000Fu) | 0x64006400u, blo, dw),
                      a_pair((w & 0x00F000F0u) | 0x54005400u, bhi, dw),
                      a_pair((w8 & 0x00F000F0u) | 0x54005400u, bhi, dw));
}
__device__ __forceinline__ __half2 half2_bits(uint32_t v) { return *reinterpret_cast<const __half2 *>(&v); }
// zero point 8: biases 1024 + 8 and 64 + 8
__device__ __forceinline__ uint4 a_word(uint32_t w, __half2 dw) {
    return a_word(w, dw, half2_bits(0x64086408u), half2_bits(0x54805480u));
}

// Two codes of word v (bytes k and k + 2, k = 0 or 1) -> f16 pair q * d_a. A code becomes an
// exact half by placing its biased byte (q + 128) under the exponent of 1024 (PRMT); subtracting
// 1152 leaves q exactly; the binary16 multiply by d_a rounds the exact product once, as the
// binary32 product rounded to binary16 would.
__device__ __forceinline__ uint32_t b_pair(uint32_t u, uint32_t sel, __half2 d2) {
    uint32_t h;
    asm("prmt.b32 %0, %1, 0x64646464, %2;" : "=r"(h) : "r"(u), "r"(sel));
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
    const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&h), bias), d2);
    return *reinterpret_cast<const uint32_t *>(&r);
}
// four codes (one word, elements e .. e+3) -> halves in the order e, e+2, e+1, e+3
__device__ __forceinline__ uint2 b_word(uint32_t v, __half2 d2) {
    const uint32_t u = v ^ 0x80808080u;   // q + 128 in each byte
    return make_uint2(b_pair(u, 0x4240u, d2), b_pair(u, 0x4341u, d2));
}

// Word w of an image block (codes 4w .. 4w+3 and 16+4w .. 16+4w+3) and the block's scale
struct ImageWord {
    uint32_t lo, hi;
    uint16_t d;
};
__device__ __forceinline__ ImageWord image_word(const int8_t *qs, const uint16_t *d, int64_t block, int w) {
    const uint32_t *src = reinterpret_cast<const uint32_t *>(qs + block * QB);
    return {ld_prev(src + w), ld_prev(src + 4 + w), ld_prev(d + block)};
}
// -> f16 q * d_a at dst's columns 2w, 2w+1 (halves 4w .. 4w+3) and 8+2w, 9+2w (halves 16+4w ..), the K order of the
// A stages
__device__ __forceinline__ void dequant_word(const ImageWord &x, int w, __half *dst) {
    const __half dah = __ushort_as_half(x.d);
    const __half2 d2 = __halves2half2(dah, dah);
    *reinterpret_cast<uint2 *>(dst + 4 * w) = b_word(x.lo, d2);
    *reinterpret_cast<uint2 *>(dst + 16 + 4 * w) = b_word(x.hi, d2);
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}


}  // namespace qk

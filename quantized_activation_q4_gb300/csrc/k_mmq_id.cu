// Routed prefill: matrix products grouped by expert with ragged sizes on a Q8_0 activation image
// (the GEMMs of minfer doc 52 "r49 A-quantize prepass shared-A dedup", section 1, over the grouped
// plan of TensorFold PR #1047 "The fix"; llama.cpp PR #117 Coverage: the image is independent of
// route ids).
//
//   y[p][n] = bf16( sum_i W_e[n][i] * x_row(p)[i] ),  W = (nibble - z) * d_w,  x = q * d_a
//
// On the 5th-generation tensor cores: operands W and x as binary16, each rounded once, binary32
// accumulation over all of K in tensor memory. (Exact operands would need W and x in two halves and
// three MMAs; the outputs are bfloat16, whose rounding is eight times the operands'.)
//
// Two kernels per call: dequant_pairs_kernel writes the planned pairs' image rows as binary16 in plan
// order (in the caller's workspace), so that an expert's pairs are consecutive rows and a pass is a
// plain tile; then mmq_id_kernel.
//
// Work items are (expert, 128-row weight tile, pass): a pass is up to 128 of the expert's pairs. An
// expert with c pairs has ceil(c / 128) passes whose sizes differ by less than 32 (qk_passes.cuh), so that
// no pass is a small remainder, and a pass of n pairs runs MMAs of N = n rounded up to 16 columns: the
// tensor work follows the ragged counts. Items are taken round-robin, passes fastest, so that the CTAs
// that run at one time share weight tiles through L2. Every CTA derives the item list from the counts.
//
// A stage is 128 K elements: A as 64 tensor-memory columns, B as two 64-column slabs. The accumulator is
// double: the next item's MMAs run while one is read.
//   warp 0:       streams the packed weights (one stage's 128 rows x 128 K per slot) by bulk copies
//   warp 1:       allocates tensor memory, issues the MMAs
//   warps 2-9:    packed nibbles -> binary16 A stages, two groups of four warps in turn
//   warps 10-17:  accumulator -> bfloat16 rows, scattered to the pairs' output rows
//   warp 18:      the pass's activation rows, a tensor copy per stage
//   warp 19:      looks the items up, up to four ahead of the epilogue (a descriptor and the pass's pair
//                 list per item), so that no other warp waits for the plan's words
//
// What bounds it: with many pairs the MMAs (8 x n / 2 cycles a stage) and, beside them, the instructions of
// the conversion, about 1100 a stage; with few pairs the conversion and the weight stream. What the steps
// there gave (gate/up of 128 experts, K 2560, 2 x 768 rows, top 8 of 512 / of 4096 rows, us):
//   - rows gathered out of the unsorted image by four-row tensor copies 394 / 1338, by 16-byte asynchronous
//     copies of six warps 239 / 714, in plan order through the workspace 212 / 476;
//   - copies and MMAs issued under elect.sync and not under a test of the lane number, which costs a loop
//     over the lanes: 177 / 433;
//   - one full and one empty barrier per stage 137 / 416 (a look at a barrier takes 90 cycles and more even
//     when its phase is complete);
//   - short bodies for the roles' loops 125 / 390: twenty warps in five roles share the instruction caches,
//     and unrolling the MMA loop over the ring cost a quarter;
//   - ring positions by additions 109 / 297: a lone warp issues a dependent instruction every five to ten
//     cycles, so a division in its loop is 200 cycles of its stage;
//   - stmatrix and 16-byte stores in the epilogue 101 / 284 (down projection 193 -> 127);
//   - the single warps' loops in one elected thread, the MMA thread looking at the next stage's barrier
//     before it issues this one's MMAs 92 / 276; eight converter warps for sixteen 88 / 242;
//   - the plan read and weights in flight while dequant_pairs_kernel runs 84 / 237 (of which that kernel takes
//     9 / 31, mostly the writing of 21 / 168 MB); a group's scales loaded once for its blocks 84 / 229.
// Those are bursts; over seconds the 4096 rows draw the GPU's 1400 W and take 266 at 1550 MHz.
// What is left: with the conversion's arithmetic taken out 73 / 197, with two MMAs a stage of eight 82 / 212, with
// both 70 / 173; the tensor pipe is 22% / 59% active, the issue slots 59% / 68%. A stage's hand-overs from role
// to role cost about 450 cycles that no arrangement tried here hides:
//   - passes of 64 pairs with six stages for few pairs per expert 5% slower; passes of up to 256 pairs (a converted
//     weight serves twice the products) with stages of 64 K 117 / 243;
//   - two pipelines with an MMA thread each, or four converter groups: the same;
//   - image rows converted once (21 MB for 168) and gathered by four-row copies from two warps' elected threads
//     108 / 352: a gather takes the copy engine 20 cycles.
// The conversion of the weights is that of the dense prefill kernel (k_mmq.cu).

#include <atomic>

#include <cuda_bf16.h>

#include "qk_internal.cuh"
#include "qk_passes.cuh"
#include "qk_tc.cuh"

namespace qk {
namespace {

constexpr int MAX_PROJ = 8;
constexpr int MAX_E = 1024;
constexpr int TM = 128;              // weight rows per item (MMA M)
constexpr int TN = PASS_MOST;        // most pairs of a pass (MMA N)
constexpr int KC = 64;               // K elements of one slab of activations (a 128-byte swizzle row)
constexpr int SK = 128;              // K elements per stage
constexpr int NS = 4;                // stages: A in tensor memory, B in shared memory
constexpr int NU = 8;                // packed-weight slots
constexpr int BOX_ROWS = 32;         // activation copies come in multiples of so many rows
constexpr int B_STAGE = TN * SK * 2; // 32 KB
constexpr int U_SLOT = Q4_UNIT_BYTES;
constexpr uint32_t A_COLS = SK / 2;  // tensor-memory columns of an A stage
constexpr uint32_t A_TMEM = 2 * TN;  // the A stages follow the two accumulators
constexpr uint32_t TMEM_COLS = 512;
constexpr int GROUPS = 2, GROUP_WARPS = 4;   // converter groups take turns at the stages
constexpr int CONV0 = 2, EPI0 = CONV0 + GROUPS * GROUP_WARPS, N_EPI = 8, ACT_WARP = EPI0 + N_EPI, ITEM_WARP = ACT_WARP + 1;
constexpr int THREADS = (ITEM_WARP + 1) * 32;
constexpr int N_READERS = 3 + GROUPS * GROUP_WARPS + N_EPI;   // warps that read an item's descriptor
constexpr int NI = 4;                // item descriptors
constexpr int EPI_BYTES = 1024;      // an epilogue warp's 16 pairs x 32 rows of bfloat16
static_assert(A_TMEM + NS * A_COLS <= TMEM_COLS, "tensor memory");
static_assert(4 * strip_unit_bytes(64) <= U_SLOT, "a weight stage fits its slot");
// a stage or slot always meets the same group, so that no barrier is waited on a phase too early
static_assert(NS % GROUPS == 0 && NU % GROUPS == 0, "rings");

struct Item {
    int e, j, rt;        // expert, projection, row tile of the projection
    int pass, passes;
};
struct Info {            // what the other warps need of an item
    int e, j, rt;        // expert, projection, row tile of the projection
    int n, first, K;     // pairs of the pass, plan position of the first; inner size
    int pad[2];
    int pair[TN];        // their pair numbers, -1 where the plan names none of this bucket
};

// shared memory: [B stages][weights][epilogue][descriptors][pass prefix][barriers][tensor-memory address,
// item count]
constexpr int OFF_U = NS * B_STAGE;
constexpr int OFF_EPI = OFF_U + NU * U_SLOT;
constexpr int OFF_INFO = OFF_EPI + N_EPI * EPI_BYTES;
constexpr int OFF_PRE = OFF_INFO + NI * (int)sizeof(Info);
constexpr int OFF_BAR = (OFF_PRE + (MAX_E + 1) * 4 + 7) / 8 * 8;
// full[NS] empty[NS] ufull[NU] uempty[NU] acc_full[2] acc_empty[2] info_full[NI] info_empty[NI] mma_done
constexpr int N_BARS = 2 * NS + 2 * NU + 2 * NI + 5;
constexpr int SMEM_BYTES = OFF_BAR + N_BARS * 8 + 8 + 1024;   // + slack to align the base to 1024
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

struct IdProj {
    const uint8_t *w;
    uint16_t *y;
    int64_t y_stride, expert_bytes;
    int N, K, chunks, rt_begin;   // rt_begin: first row tile of this projection in the launch
};
struct IdArgs {
    // activations [pairs][K] binary16 in plan order, seen as [K / 64][pairs][64]: boxes of two 64-column
    // slabs x 32, 64, 96 or 128 rows, swizzled
    CUtensorMap bmap[4];
    const int32_t *counts, *offsets, *items;
    int pairs, E, n_proj, row_tiles;
    IdProj p[MAX_PROJ];
};

__device__ __forceinline__ int clamped_count(const IdArgs &a, int e) {
    const int c = __ldcg(a.counts + e);
    return c < 0 ? 0 : (c > a.pairs ? a.pairs : c);
}
// Item tau: its expert is the last e with pre[e] <= tau / row_tiles (pre: prefix of the pass counts).
__device__ __forceinline__ Item item_of(const IdArgs &a, const int *pre, int tau) {
    const int q = tau / a.row_tiles;
    int lo = 0, hi = a.E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= q)
            lo = mid;
        else
            hi = mid;
    }
    Item t;
    t.e = lo;
    t.passes = pre[lo + 1] - pre[lo];
    const int local = tau - pre[lo] * a.row_tiles, r = local / t.passes;
    t.pass = local - r * t.passes;
    t.j = 0;
    while (t.j + 1 < a.n_proj && r >= a.p[t.j + 1].rt_begin) t.j++;
    t.rt = r - a.p[t.j].rt_begin;
    return t;
}
// Pairs of the item's pass: `first` is their position in the plan, n (1..TN) their number.
struct Pairs {
    int64_t first;
    int n;
};
__device__ __forceinline__ Pairs pairs_of(const IdArgs &a, const Item &t) {
    const PassRange r = pass_range(clamped_count(a, t.e), t.passes, t.pass);
    return {(int64_t)__ldcg(a.offsets + t.e) + r.start, r.n};
}
// The pair at plan position pos, -1 outside the plan or the bucket (a plan from elsewhere).
__device__ __forceinline__ int pair_at(const IdArgs &a, int64_t pos) {
    if (pos < 0 || pos >= a.pairs) return -1;
    const int p = __ldcg(a.items + pos);
    return p >= 0 && p < a.pairs ? p : -1;
}

// One lane of a converged warp. Tensor copies, MMAs and commits take their operands from uniform
// registers: under elect.sync the compiler issues them directly (an MMA about 17 cycles), under a
// test of the lane number in a loop over the lanes (about 150).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// Whether the phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t a, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    return ok != 0;
}
// A whole warp's wait: every lane gets the same answer. A phase that is complete costs one look.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
// Both of two barriers; their looks overlap.
__device__ __forceinline__ bool warp_wait2(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1) {
    const bool d0 = mbar_test(bar0, parity0), d1 = mbar_test(bar1, parity1);
    if (__all_sync(0xffffffffu, d0 && d1)) return true;
    const bool w = mbar_wait(bar0, parity0) && mbar_wait(bar1, parity1);
    return __all_sync(0xffffffffu, w);
}
// A position in a ring of N entries: barriers 8 bytes apart, the parity of the phase that is filled
// next. Single warps run these loops, a dependent instruction every five cycles or so: the positions
// advance by additions. An entry's empty barrier is waited for with parity ^ 1: the first round passes.
struct Ring {
    uint32_t at, parity;
    __device__ __forceinline__ void next(int n, int step = 1) {
        at += step;
        if (at >= (uint32_t)n) {
            at -= n;
            parity ^= 1;
        }
    }
};
// D += A x B (see tc_mma)
__device__ __forceinline__ void tc_mma_add(uint32_t tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.eq.u32 p, 0, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem),
        "r"(a_tmem), "l"(b), "r"(idesc)
        : "memory");
}
// a box at column 0, row y, slab z
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int y, int z, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(mbar)
        : "memory");
}
// 16 accumulator columns of this warp's 32 rows to bfloat16 in shared memory, 64 bytes per column: with
// the 16x256b shape lane 4g + t holds rows g and g + 8 of columns 2t, 2t+1 (and 8+2t, 9+2t), the fragments
// that stmatrix transposes, so that 8 rows of a column are 16 consecutive bytes. Piece c (rows 8c..) of
// column j is stored at place c ^ (j / 2 % 4): no two rows of a matrix share banks.
__device__ __forceinline__ uint32_t pack_bf16(uint32_t lo, uint32_t hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
    return r;
}
__device__ __forceinline__ void columns_to_smem(uint32_t taddr, uint32_t buf, int lane) {
    uint32_t v[16];
#pragma unroll
    for (int h = 0; h < 2; h++)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[8 * h]), "=r"(v[8 * h + 1]), "=r"(v[8 * h + 2]), "=r"(v[8 * h + 3]), "=r"(v[8 * h + 4]),
                       "=r"(v[8 * h + 5]), "=r"(v[8 * h + 6]), "=r"(v[8 * h + 7])
                     : "r"(taddr + (uint32_t)(h << 20)));   // lanes 0-15, then 16-31
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int c = 0; c < 2; c++) {   // columns 8c .. 8c+7; lane 8m + j addresses piece m of column j
        const int col = 8 * c + (lane & 7);
        const uint32_t dst = buf + col * 64 + (((lane >> 3) ^ ((col >> 1) & 3)) << 4);
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(dst),
                     "r"(pack_bf16(v[4 * c], v[4 * c + 1])), "r"(pack_bf16(v[4 * c + 2], v[4 * c + 3])),
                     "r"(pack_bf16(v[8 + 4 * c], v[8 + 4 * c + 1])), "r"(pack_bf16(v[8 + 4 * c + 2], v[8 + 4 * c + 3]))
                     : "memory");
    }
}

// The converters' words of one 32-column block for a warp's 32 rows: lane (g, t) gets word t of rows
// g, g+8, 16+g, 24+g, their scales and the biases that hold the zero points.
template <int WT>
struct RowHeads {
    __half2 dw[4], blo[4], bhi[4];
};
template <int WT>
__device__ __forceinline__ void load_heads(const uint8_t *unit, int quad, int jb, int gq, RowHeads<WT> &h) {
    if (WT == QK_W_Q4_0) {
        const uint2 sc = *reinterpret_cast<const uint2 *>(unit + 8192 + jb * 256 + gq * 32 + quad * 8);
        const __half2 s01 = half2_bits(sc.x), s23 = half2_bits(sc.y);
        h.dw[0] = __low2half2(s01);
        h.dw[1] = __high2half2(s01);
        h.dw[2] = __low2half2(s23);
        h.dw[3] = __high2half2(s23);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            h.blo[i] = half2_bits(0x64086408u);
            h.bhi[i] = half2_bits(0x54805480u);
        }
    } else {
        constexpr int G = WT == QK_W_Q4_G64 ? 64 : 128;
        const uint4 hd = *reinterpret_cast<const uint4 *>(unit + quad * strip_unit_bytes(G) + STRIP_DATA +
                                                          128 * (jb * QB / G) + 16 * gq);
        const uint32_t v[4] = {hd.x, hd.y, hd.z, hd.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            h.dw[i] = __low2half2(half2_bits(v[i]));
            const __half2 z8 = __high2half2(half2_bits(v[i]));   // z - 8, an integer: both sums are exact
            h.blo[i] = __hadd2(half2_bits(0x64086408u), z8);
            h.bhi[i] = __hadd2(half2_bits(0x54805480u), z8);
        }
    }
}
template <int WT>
__device__ __forceinline__ uint4 load_words(const uint8_t *unit, int quad, int jb, int lane) {
    if (WT == QK_W_Q4_0)
        return *reinterpret_cast<const uint4 *>(unit + jb * Q4_BLOCK_STRIDE + quad * 512 + lane * 16);
    constexpr int G = WT == QK_W_Q4_G64 ? 64 : 128;
    return *reinterpret_cast<const uint4 *>(unit + quad * strip_unit_bytes(G) + jb * 512 + lane * 16);
}

// A warp per plan position: row pos of the activations from the image row of the pair there, eight
// blocks per step (lane l: word l & 3 of block l / 4).
__global__ void __launch_bounds__(256) dequant_pairs_kernel(const int8_t *qs, const uint16_t *d, int64_t row_blocks,
                                                            const int32_t *offsets, const int32_t *items, int E,
                                                            int pairs, int k, int per_pair, int kb, int64_t pitch,
                                                            __half *__restrict__ B) {
    pdl_wait();
    pdl_trigger();   // after the wait: when mmq_id_kernel starts, the kernel that wrote the plan has completed
    const int pos = blockIdx.x * 8 + (threadIdx.x >> 5), w = threadIdx.x & 3, b0 = (threadIdx.x & 31) >> 2;
    if (pos >= pairs || pos >= ld_prev(offsets + E)) return;   // positions past the plan hold no pair
    const int p = ld_prev(items + pos);
    if (p < 0 || p >= pairs) return;
    const int64_t first = (per_pair ? p : p / k) * row_blocks;
    __half *dst = B + pos * pitch;
    for (int b = b0; b < kb; b += 32) {   // four loads in flight
        ImageWord x[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (b + 8 * i < kb) x[i] = image_word(qs, d, first + b + 8 * i, w);
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (b + 8 * i < kb) dequant_word(x[i], w, dst + (int64_t)(b + 8 * i) * QB);
    }
}

template <int WT>
__global__ void __launch_bounds__(THREADS, 1) mmq_id_kernel(const __grid_constant__ IdArgs a) {
    constexpr bool GROUPED = WT != QK_W_Q4_0;
    constexpr int STRIP = strip_unit_bytes(WT == QK_W_Q4_G64 ? 64 : 128);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t full = sbase + OFF_BAR, empty = full + NS * 8, ufull = empty + NS * 8, uempty = ufull + NU * 8,
                   acc_full = uempty + NU * 8, acc_empty = acc_full + 16, info_full = acc_empty + 16,
                   info_empty = info_full + 8 * NI, mma_done = info_empty + 8 * NI;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_BAR + N_BARS * 8);
    int *n_items = reinterpret_cast<int *>(tmem_slot + 1);
    Info *info = reinterpret_cast<Info *>(smem + OFF_INFO);
    int *pre = reinterpret_cast<int *>(smem + OFF_PRE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; s++) {
            mbar_init(full + 8 * s, GROUP_WARPS + 1); // its group's converter warps; the activation warp, with the bytes
            mbar_init(empty + 8 * s, 1);              // the MMA commit
        }
        for (int u = 0; u < NU; u++) {
            mbar_init(ufull + 8 * u, 1);              // the weight warp, with the bytes
            mbar_init(uempty + 8 * u, GROUP_WARPS);
        }
        for (int h = 0; h < 2; h++) {
            mbar_init(acc_full + 8 * h, 1);         // the MMA commit after an item's last stage
            mbar_init(acc_empty + 8 * h, N_EPI);    // the epilogue warps, once they have read it
        }
        for (int i = 0; i < NI; i++) {
            mbar_init(info_full + 8 * i, 1);        // the item warp
            mbar_init(info_empty + 8 * i, N_READERS);
        }
        mbar_init(mma_done, 1);               // the MMA thread's last commit
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_trigger();
    if (warp == 0) {
        // prefix of the experts' pass counts: lane l sums experts l * per .. l * per + per - 1. Plans of
        // this bucket have at most pairs / TN + E passes; counts with more are refused (fault bit 1).
        const int per = (a.E + 31) / 32, e0 = min(a.E, lane * per), e1 = min(a.E, e0 + per);
        int64_t sum = 0;
        for (int e = e0; e < e1; e++) sum += passes_of(clamped_count(a, e));
        int64_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
        const bool sound = total <= a.pairs / TN + a.E;
        int64_t at = incl - sum;
        for (int e = e0; e < e1; e++) {
            pre[e] = sound ? (int)at : 0;
            at += passes_of(clamped_count(a, e));
        }
        if (lane == 31) {
            pre[a.E] = sound ? (int)total : 0;
            *n_items = sound ? (int)total * a.row_tiles : 0;
            if (!sound) atomicOr(&g_tc_faults, 2u);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int items = *n_items;

    // Item i of this CTA (items blockIdx.x + i * gridDim.x): entry i % NI of the descriptor ring. A
    // warp waits for it, and arrives on info_empty when it needs it no more.
    auto await_info = [&](int i) { return warp_wait(info_full + 8 * (i % NI), (i / NI) & 1); };
    auto release_info = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(info_empty + 8 * (i % NI));
    };
    const int mine = items > (int)blockIdx.x ? (items - (int)blockIdx.x + G - 1) / G : 0;   // this CTA's items

    if (warp == ITEM_WARP) {   // ---------------- items
        for (int i = 0; i < mine; i++) {
            const Item t = item_of(a, pre, blockIdx.x + i * G);
            const Pairs pr = pairs_of(a, t);
            int p[TN / 32];
#pragma unroll
            for (int j = 0; j < TN / 32; j++)
                p[j] = 32 * j + lane < pr.n ? pair_at(a, pr.first + 32 * j + lane) : -1;
            if (i >= NI && !warp_wait(info_empty + 8 * (i % NI), ((i / NI) - 1) & 1)) break;
            Info &f = info[i % NI];
#pragma unroll
            for (int j = 0; j < TN / 32; j++) f.pair[32 * j + lane] = p[j];
            if (lane == 0) {
                f.e = t.e;
                f.j = t.j;
                f.rt = t.rt;
                f.n = pr.n;
                f.K = a.p[t.j].K;
                // rows outside the plan's read as zeros (a plan from elsewhere: none of them is stored)
                f.first = (int)(pr.first < -TN ? -TN : (pr.first > a.pairs ? a.pairs : pr.first));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(info_full + 8 * (i % NI));
        }
    } else if (warp == 0) {   // ---------------- weights
        if (elect_one()) {
            Ring u = {0, 0};
            uint32_t issued = 0;   // weight stages issued by this CTA
            bool ok = true;
            for (int i = 0; i < mine && ok; i++) {
                if (!mbar_wait(info_full + 8 * (i % NI), (i / NI) & 1)) break;
                const Info &f = info[i % NI];
                const IdProj &P = a.p[f.j];
                const int chunks = P.chunks, strips = GROUPED ? min(4, (P.N - f.rt * TM + STRIP_ROWS - 1) / STRIP_ROWS) : 1;
                constexpr uint32_t PIECE = GROUPED ? STRIP : Q4_UNIT_BYTES;   // one strip's or the whole tile's stage
                const int64_t row_bytes = (int64_t)chunks * PIECE;            // strips are this far apart
                const uint8_t *w = P.w + f.e * P.expert_bytes + (int64_t)f.rt * (GROUPED ? 4 : 1) * row_bytes;
                mbar_arrive(info_empty + 8 * (i % NI));
                for (int kc = 0; kc < chunks; kc++, w += PIECE, issued++) {
                    if (!mbar_wait(uempty + 8 * u.at, u.parity ^ 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + OFF_U + u.at * U_SLOT, bar = ufull + 8 * u.at;
                    mbar_expect_tx(bar, strips * PIECE);
                    bulk_g2s(dst, w, PIECE, bar);
                    if (GROUPED) {
                        if (strips > 1) bulk_g2s(dst + PIECE, w + row_bytes, PIECE, bar);
                        if (strips > 2) bulk_g2s(dst + 2 * PIECE, w + 2 * row_bytes, PIECE, bar);
                        if (strips > 3) bulk_g2s(dst + 3 * PIECE, w + 3 * row_bytes, PIECE, bar);
                    }
                    u.next(NU);
                }
            }
            // Every copy this thread issued has landed before the CTA can exit, also after a wait above ran
            // out (a barrier whose phase completed long ago passes at once; a wait that runs out here ends
            // the drain).
            for (uint32_t x = issued > NU ? issued - NU : 0; x < issued; x++)
                if (!mbar_wait(ufull + 8 * (x % NU), (x / NU) & 1u)) break;
        }
        __syncwarp();
    } else if (warp == ACT_WARP) {   // ---------------- activations
        if (elect_one()) {
            pdl_wait();   // the binary16 rows; in every CTA, so that this kernel completes after that one
            Ring r = {0, 0};
            uint32_t issued = 0;   // stages filled by this CTA
            bool ok = true;
            for (int i = 0; i < mine && ok; i++) {
                if (!mbar_wait(info_full + 8 * (i % NI), (i / NI) & 1)) break;
                const Info &f = info[i % NI];
                const int slabs = (f.K + KC - 1) / KC, first = f.first, boxes = (f.n + BOX_ROWS - 1) / BOX_ROWS;
                const CUtensorMap *map = &a.bmap[boxes - 1];
                const uint32_t bytes = boxes * BOX_ROWS * SK * 2;   // a slab past K counts, filled with zeros
                mbar_arrive(info_empty + 8 * (i % NI));
                for (int slab = 0; slab < slabs; slab += 2, issued++) {
                    if (!mbar_wait(empty + 8 * r.at, r.parity ^ 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = full + 8 * r.at;
                    mbar_expect_tx(bar, bytes);
                    tma_3d(sbase + r.at * B_STAGE, map, first, slab, bar);
                    r.next(NS);
                }
            }
            // as for the weights: all copies have landed (a stage whose converters stopped never completes:
            // the wait runs out, long after its copies)
            for (uint32_t x = issued > NS ? issued - NS : 0; x < issued; x++)
                if (!mbar_wait(full + 8 * (x % NS), (x / NS) & 1u)) break;
        }
        __syncwarp();
    } else if (warp == 1) {   // ---------------- MMA issue (one elected thread, always the same)
        if (elect_one()) {
            Ring r = {0, 0};
            bool ok = true, ready = false;
            for (int i = 0; i < mine && ok; i++) {
                const uint32_t entry = 8 * (i % NI), side = 8 * (i & 1);
                if (!mbar_wait(info_full + entry, (i / NI) & 1)) break;
                const int n = info[i % NI].n, K = info[i % NI].K;
                mbar_arrive(info_empty + entry);
                const uint32_t idesc = mma_idesc((n + 15) & ~15), acc = tmem + (i & 1) * TN;
                const uint32_t slab16 = (n + BOX_ROWS - 1) / BOX_ROWS * (BOX_ROWS * KC * 2 / 16);   // a slab's rows, in descriptor units
                if (!mbar_wait(acc_empty + side, ((i >> 1) & 1) ^ 1)) break;
                for (int left = K; left > 0; left -= SK) {   // nothing past K enters the sum
                    if (!ready && !mbar_wait(full + 8 * r.at, r.parity)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = r.at;
                    r.next(NS);
                    ready = mbar_test(full + 8 * r.at, r.parity);   // the next stage's look overlaps this one's MMAs
                    tc_fence_after();
                    // a descriptor's address field counts 16-byte units
                    const uint32_t ta = tmem + A_TMEM + at * A_COLS;
                    const uint64_t bd = sdesc(sbase + at * B_STAGE);
                    tc_mma(acc, ta, bd, idesc, left != K);
                    if (left >= SK) {
#pragma unroll
                        for (int ks = 1; ks < SK / 16; ks++)
                            tc_mma_add(acc, ta + 8 * ks, bd + (uint64_t)((ks >> 2) * slab16 + 2 * (ks & 3)), idesc);
                    } else {
#pragma unroll 1
                        for (int ks = 1; 16 * ks < left; ks++)
                            tc_mma_add(acc, ta + 8 * ks, bd + (uint64_t)((ks >> 2) * slab16 + 2 * (ks & 3)), idesc);
                    }
                    tc_commit(empty + 8 * at);
                    if (left <= SK) tc_commit(acc_full + side);
                }
            }
            tc_commit(mma_done);   // every MMA issued here is complete before the tensor memory is freed
            mbar_wait(mma_done, 0u);
        }
        __syncwarp();
    } else if (warp < EPI0) {   // ---------------- A conversion into tensor memory
        // lanes 32 (warp % 4) .. +31 of tensor memory are tile rows 32 (warp % 4) ..; a warp takes them in its
        // group's stages
        const int quad = warp & 3, group = (warp - CONV0) / GROUP_WARPS, gq = lane >> 2;
        const uint32_t abase = tmem + ((uint32_t)(32 * quad) << 16) + A_TMEM;
        Ring ra = {(uint32_t)group, 0}, u = {(uint32_t)group, 0};
        int ahead = group;   // stages until this group's next one
        bool ok = true;
        for (int i = 0; i < mine && ok; i++) {
            if (!await_info(i)) break;
            const int chunks = (info[i % NI].K + SK - 1) / SK;
            release_info(i);
            for (; ahead < chunks; ahead += GROUPS) {
                ok = warp_wait2(ufull + 8 * u.at, u.parity, empty + 8 * ra.at, ra.parity ^ 1);
                if (!ok) break;
                tc_fence_after();
                const uint8_t *unit = smem + OFF_U + u.at * U_SLOT;
                constexpr int HEAD_BLOCKS = WT == QK_W_Q4_0 ? 1 : WT == QK_W_Q4_G64 ? 2 : 4;   // blocks of one scale
                RowHeads<WT> hd;
#pragma unroll
                for (int jb = 0; jb < 4; jb++) {
                    const uint4 wv = load_words<WT>(unit, quad, jb, lane);
                    if (jb % HEAD_BLOCKS == 0) load_heads<WT>(unit, quad, jb, gq, hd);
                    const uint4 a0 = a_word(wv.x, hd.dw[0], hd.blo[0], hd.bhi[0]);
                    const uint4 a1 = a_word(wv.y, hd.dw[1], hd.blo[1], hd.bhi[1]);
                    const uint4 a2 = a_word(wv.z, hd.dw[2], hd.blo[2], hd.bhi[2]);
                    const uint4 a3 = a_word(wv.w, hd.dw[3], hd.blo[3], hd.bhi[3]);
                    const uint32_t base = abase + ra.at * A_COLS + 16 * jb;
                    asm volatile(
                        "tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(base),
                        "r"(a0.x), "r"(a0.y), "r"(a1.x), "r"(a1.y), "r"(a0.z), "r"(a0.w), "r"(a1.z), "r"(a1.w)
                        : "memory");
                    asm volatile(
                        "tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(base + (16u << 16)),
                        "r"(a2.x), "r"(a2.y), "r"(a3.x), "r"(a3.y), "r"(a2.z), "r"(a2.w), "r"(a3.z), "r"(a3.w)
                        : "memory");
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {   // one arrival per warp: a lane's arrivals on one barrier go one by one
                    mbar_arrive(full + 8 * ra.at);
                    mbar_arrive(uempty + 8 * u.at);
                }
                ra.next(NS, GROUPS);
                u.next(NU, GROUPS);
            }
            ahead -= chunks;
        }
    } else {   // ---------------- epilogue (accumulator lane = weight row, column = pair)
        const int quad = warp & 3, c0 = ((warp - EPI0) >> 2) * (TN / 2), piece = lane & 3;
        const uint32_t buf = sbase + OFF_EPI + (warp - EPI0) * EPI_BYTES;
        for (int i = 0; i < mine; i++) {
            if (!warp_wait2(info_full + 8 * (i % NI), (i / NI) & 1, acc_full + 8 * (i & 1), (i >> 1) & 1)) break;
            tc_fence_after();
            const Info &f = info[i % NI];
            const IdProj &P = a.p[f.j];
            const int n = min(f.n - c0, TN / 2), row = f.rt * TM + quad * 32 + 8 * piece, rows = P.N - row;
            const bool wide = rows >= 8 && ((reinterpret_cast<uintptr_t>(P.y) | (uintptr_t)(P.y_stride * 2)) & 15) == 0;
            uint16_t *yr = P.y + row;
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)((i & 1) * TN + c0);
#pragma unroll 1   // a short body: the roles share the SM's instruction caches
            for (int q = 0; q < n; q += 16) {
                __syncwarp();   // the previous columns have been read
                columns_to_smem(taddr + q, buf, lane);
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 16; c += 8) {
                    const int col = c + (lane >> 2), id = f.pair[c0 + q + col];   // -1 past the pass's pairs
                    uint32_t x[4];
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                 : "r"(buf + col * 64 + ((piece ^ ((col >> 1) & 3)) << 4)));
                    if (id < 0) continue;
                    uint16_t *dst = yr + id * P.y_stride;
                    if (wide) {
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            if (e < rows) dst[e] = (uint16_t)(x[e >> 1] >> (16 * (e & 1)));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + 8 * (i & 1));
            release_info(i);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                     : "memory");
}

template <int WT>
qk_status launch_type(const IdArgs &a, cudaStream_t s) {
    constexpr int MAXDEV = 64;
    static std::atomic<bool> set[MAXDEV];   // the kernel's attribute, once per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= MAXDEV || !set[dev].load(std::memory_order_relaxed))) {
        e = cudaFuncSetAttribute(mmq_id_kernel<WT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        if (e == cudaSuccess && dev >= 0 && dev < MAXDEV) set[dev].store(true, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "mmq_id: shared memory attribute: %s", cudaGetErrorString(e));
    return launch_pdl("mmq_id", mmq_id_kernel<WT>, dim3((unsigned)sm_count()), dim3(THREADS), (size_t)SMEM_BYTES, s, a);
}

}  // namespace

// columns of an activation row in the workspace: whole 64-column slabs
static int64_t act_pitch(int64_t kmax) { return (kmax + KC - 1) / KC * KC; }
int64_t mmq_id_workspace_bytes(int64_t pairs, int64_t kmax) { return pairs * act_pitch(kmax) * 2; }

qk_status read_mmq_id_faults(uint32_t *faults) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tc_faults, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_tc_faults, &zero, sizeof zero);
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "qk_device_faults: %s", cudaGetErrorString(e));
    *faults = v;
    return QK_OK;
}

qk_status launch_mmq_id(const int8_t *qs, const uint16_t *d, int64_t row_blocks, int rows, int k,
                        int n_proj, const qk_proj_id16 *projs, const int32_t *counts, const int32_t *offsets,
                        const int32_t *items, bool per_pair, void *ws, cudaStream_t s) {
    int64_t kmax = 0;
    for (int j = 0; j < n_proj; j++) kmax = projs[j].K > kmax ? projs[j].K : kmax;
    IdArgs a = {};
    const int pairs = rows * k, kb = (int)(kmax / QB);
    const int64_t pitch = act_pitch(kmax), slabs = pitch / KC;
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return fail(QK_ERR_CUDA, "mmq_id: cuTensorMapEncodeTiled is not available");
    for (int h = 0; h < 4 && BOX_ROWS * h < pairs; h++) {   // no pass needs a larger box
        const cuuint64_t dims[3] = {KC, (cuuint64_t)pairs, (cuuint64_t)slabs};
        const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, KC * 2};
        const cuuint32_t box[3] = {KC, (cuuint32_t)(BOX_ROWS * (h + 1)), 2}, estr[3] = {1, 1, 1};
        const CUresult r = enc(&a.bmap[h], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, ws, dims, strides, box, estr,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return fail(QK_ERR_CUDA, "mmq_id: tensor map encoding failed (%d)", (int)r);
    }
    qk_status st = launch_pdl("mmq_id_dequant", dequant_pairs_kernel, dim3((unsigned)ceil_div(pairs, 8)),
                              dim3(256), 0, s, qs, d, row_blocks, offsets, items, (int)projs[0].n_experts, pairs, k,
                              (int)per_pair, kb, pitch, static_cast<__half *>(ws));
    if (st != QK_OK) return st;
    a.counts = counts;
    a.offsets = offsets;
    a.items = items;
    a.pairs = pairs;
    a.E = projs[0].n_experts;
    for (int wt = QK_W_Q4_0; wt <= QK_W_Q4_G128; wt++) {   // one launch per weight type present
        a.n_proj = 0;
        a.row_tiles = 0;
        for (int j = 0; j < n_proj; j++) {
            if (projs[j].wtype != wt) continue;
            IdProj &p = a.p[a.n_proj++];
            p.w = static_cast<const uint8_t *>(projs[j].w);
            p.y = projs[j].y;
            p.y_stride = projs[j].y_stride;
            p.N = (int)projs[j].N;
            p.K = (int)projs[j].K;
            p.chunks = (int)ceil_div(p.K, UNIT_COLS);
            p.expert_bytes = packed_bytes(wt, p.N, p.K);
            p.rt_begin = a.row_tiles;
            a.row_tiles += (int)ceil_div(p.N, TM);
        }
        if (a.n_proj == 0) continue;
        st = wt == QK_W_Q4_0     ? launch_type<QK_W_Q4_0>(a, s)
             : wt == QK_W_Q4_G64 ? launch_type<QK_W_Q4_G64>(a, s)
                                 : launch_type<QK_W_Q4_G128>(a, s);
        if (st != QK_OK) return st;
    }
    return QK_OK;
}

}  // namespace qk

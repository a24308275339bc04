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
// Two kernels per call: dequant_b writes the image as binary16 rows (in the caller's workspace, once,
// read by every weight row tile of every expert that a row goes to), then mmq_id_kernel.
//
// Work items are (expert, 128-row weight tile, pass): a pass is up to 256 of the expert's pairs. An
// expert with c pairs has ceil(c / 256) passes of nearly equal size, so that no pass is a small
// remainder, and a pass of n pairs runs MMAs of N = n rounded up to 16 columns: the tensor work follows
// the ragged counts. Items are taken round-robin, passes fastest, so that the CTAs that run at one
// time share weight tiles through L2. Every CTA derives the item list from the counts.
//
//   warp 0:       TMA: the packed weights of a stage (128 rows x 128 K) by bulk copies, and the pass's
//                 activation rows by four-row gathers (each lane holds the row numbers of its groups)
//   warp 1:       allocates tensor memory, issues the MMAs (one thread)
//   warps 2-9:    packed nibbles -> binary16 A stages in tensor memory
//   warps 10-25:  accumulator -> bfloat16 rows, scattered to the pairs' output rows
// The stage layout, the conversion and the barriers are those of the dense prefill kernel (k_mmq.cu).

#include <cuda_bf16.h>

#include "qk_internal.cuh"
#include "qk_tc.cuh"

namespace qk {
namespace {

constexpr int MAX_PROJ = 8;
constexpr int MAX_E = 1024;
constexpr int TM = 128;              // weight rows per item (MMA M)
constexpr int TN = 256;              // most pairs of a pass (MMA N)
constexpr int KC = 64;               // K elements of one activation box (a 128-byte swizzle row)
constexpr int SK = 128;              // K elements per stage
constexpr int NS = 3;                // stages (A in tensor memory, B in shared memory)
constexpr int NU = 3;                // packed-weight slots
constexpr int PF = 10;               // stages of weights prefetched into L2 ahead
constexpr int B_BOX = TN * KC * 2;   // 32 KB
constexpr int B_TILE = TN * SK * 2;  // 64 KB
constexpr int U_SLOT = Q4_UNIT_BYTES;
constexpr uint32_t A_COLS = SK / 2;
constexpr uint32_t A_TMEM = TN;      // A stages follow the accumulator
constexpr uint32_t TMEM_COLS = 512;
constexpr int EPI0 = 10, N_EPI = 16;
constexpr int THREADS = (EPI0 + N_EPI) * 32;
static_assert(A_TMEM + NS * A_COLS <= TMEM_COLS, "tensor memory");
static_assert(4 * strip_unit_bytes(64) <= U_SLOT, "a weight stage fits its slot");

// shared memory: [B tiles][weights][barriers][tensor-memory address, item count][pass prefix]
constexpr int OFF_U = NS * B_TILE;
constexpr int OFF_BAR = OFF_U + NU * U_SLOT;
// full_a[NS] full_b[NS] empty[NS] ufull[NU] uempty[NU] acc_full acc_empty mma_done
constexpr int N_BARS = 3 * NS + 2 * NU + 3;
constexpr int OFF_PRE = OFF_BAR + N_BARS * 8 + 16;
constexpr int SMEM_BYTES = OFF_PRE + (MAX_E + 1) * 4 + 1024;   // + slack to align the base to 1024
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

struct IdProj {
    const uint8_t *w;
    uint16_t *y;
    int64_t y_stride, expert_bytes;
    int N, K, chunks, rt_begin;   // rt_begin: first row tile of this projection in the launch
};
struct IdArgs {
    CUtensorMap bmap;             // activations [image rows][K] binary16, box 64 x 1, 128-byte swizzle
    const int32_t *counts, *offsets, *items;
    int pairs, k, E, per_pair, n_proj, row_tiles;
    IdProj p[MAX_PROJ];
};

struct Item {
    int e, j, rt;     // expert, projection, row tile of the projection
    int pass, passes;
    int nkc;          // stages
};
__device__ __forceinline__ int clamped_count(const IdArgs &a, int e) {
    const int c = __ldg(a.counts + e);
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
    t.nkc = a.p[t.j].chunks;
    return t;
}
// Pairs of the item's pass: `first` is their position in the plan, n > 0 their number.
struct Pairs {
    int64_t first;
    int n;
};
__device__ __forceinline__ Pairs pairs_of(const IdArgs &a, const Item &t) {
    const int cnt = clamped_count(a, t.e);
    const int tn = ((cnt + t.passes - 1) / t.passes + 15) & ~15;   // <= 256: passes = ceil(cnt / 256)
    const int start = t.pass * tn;
    return {(int64_t)__ldg(a.offsets + t.e) + start, min(tn, cnt - start)};
}
// The pair at plan position pos, -1 outside the plan or the bucket (a plan from elsewhere).
__device__ __forceinline__ int pair_at(const IdArgs &a, int64_t pos) {
    if (pos < 0 || pos >= a.pairs) return -1;
    const int p = __ldg(a.items + pos);
    return p >= 0 && p < a.pairs ? p : -1;
}

// A whole warp's wait: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int x, int4 r, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(mbar)
        : "memory");
}
// 32 accumulator columns of this warp's lane quarter, packed to bfloat16 pairs of columns
__device__ __forceinline__ void load_columns(uint32_t taddr, uint32_t h[16]) {
    uint32_t v[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; i++)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[i]) : "f"(__uint_as_float(v[2 * i + 1])), "f"(__uint_as_float(v[2 * i])));
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

template <int WT>
__global__ void __launch_bounds__(THREADS, 1) mmq_id_kernel(const __grid_constant__ IdArgs a) {
    constexpr bool GROUPED = WT != QK_W_Q4_0;
    constexpr int STRIP = strip_unit_bytes(WT == QK_W_Q4_G64 ? 64 : 128);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t full_a = sbase + OFF_BAR, full_b = full_a + NS * 8, empty = full_b + NS * 8;
    const uint32_t ufull = empty + NS * 8, uempty = ufull + NU * 8, acc_full = uempty + NU * 8,
                   acc_empty = acc_full + 8, mma_done = acc_empty + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_BAR + N_BARS * 8);
    int *n_items = reinterpret_cast<int *>(tmem_slot + 1);
    int *pre = reinterpret_cast<int *>(smem + OFF_PRE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; s++) {
            mbar_init(full_a + 8 * s, 256);   // the eight converter warps
            mbar_init(full_b + 8 * s, 1);     // the producer, with the bytes
            mbar_init(empty + 8 * s, 1);      // the MMA commit
        }
        for (int u = 0; u < NU; u++) {
            mbar_init(ufull + 8 * u, 1);
            mbar_init(uempty + 8 * u, 256);
        }
        mbar_init(acc_full, 1);             // the MMA commit after an item's last stage
        mbar_init(acc_empty, N_EPI * 32);   // the epilogue warps, once they have read it
        mbar_init(mma_done, 1);             // the MMA thread's last commit
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_trigger();
    pdl_wait();   // the plan and the binary16 rows come from the kernels before
    if (warp == 0) {
        // prefix of the experts' pass counts: lane l sums experts l * per .. l * per + per - 1. Plans of
        // this bucket have at most pairs / 256 + E passes; counts with more are refused (fault bit 1).
        const int per = (a.E + 31) / 32, e0 = min(a.E, lane * per), e1 = min(a.E, e0 + per);
        int64_t sum = 0;
        for (int e = e0; e < e1; e++) sum += (clamped_count(a, e) + TN - 1) / TN;
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
            at += (clamped_count(a, e) + TN - 1) / TN;
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

    if (warp == 0) {   // ---------------- producer
        uint32_t g = 0, gu = 0;   // activation stages and weight stages issued by this CTA
        bool ok = true;
        // stage kc's weights of an item into L2
        auto prefetch = [&](const Item &t, int kc) {
            const IdProj &P = a.p[t.j];
            const uint8_t *w = P.w + t.e * P.expert_bytes;
            if (GROUPED) {
                const int strip = 4 * t.rt + lane;
                if (lane < 4 && strip * STRIP_ROWS < P.N)
                    prefetch_l2(w + ((int64_t)strip * P.chunks + kc) * STRIP, STRIP);
            } else if (lane == 0) {
                prefetch_l2(w + ((int64_t)t.rt * P.chunks + kc) * Q4_UNIT_BYTES, Q4_UNIT_BYTES);
            }
        };
        Item next = {};
        if ((int)blockIdx.x < items) {
            next = item_of(a, pre, blockIdx.x);
            for (int kc = 0; kc < PF && kc < next.nkc; kc++) prefetch(next, kc);
        }
        for (int tau = blockIdx.x; tau < items && ok; tau += G) {
            const Item t = next;
            const bool more = tau + G < items;
            if (more) next = item_of(a, pre, tau + G);
            const IdProj &P = a.p[t.j];
            const uint8_t *w = P.w + t.e * P.expert_bytes;
            const Pairs pr = pairs_of(a, t);
            const int groups = ((pr.n + 15) & ~15) / 4;   // four rows each; rows past n repeat the last one
            int4 r[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                int v[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int p = max(0, pair_at(a, pr.first + min(4 * (lane + 32 * h) + i, pr.n - 1)));
                    v[i] = a.per_pair ? p : p / a.k;
                }
                r[h] = make_int4(v[0], v[1], v[2], v[3]);
            }
            const int strips = GROUPED ? min(4, (P.N - t.rt * TM + STRIP_ROWS - 1) / STRIP_ROWS) : 0;
            for (int kc = 0; kc < t.nkc; kc++, g++) {
                const uint32_t s = g % NS, us = gu % NU;
                if (gu >= NU && !warp_wait(uempty + 8 * us, ((gu / NU) - 1) & 1u)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_expect_tx(ufull + 8 * us, GROUPED ? strips * STRIP : Q4_UNIT_BYTES);
                __syncwarp();
                if (GROUPED) {
                    if (lane < strips)
                        bulk_g2s(sbase + OFF_U + us * U_SLOT + lane * STRIP,
                                 w + ((int64_t)(4 * t.rt + lane) * P.chunks + kc) * STRIP, STRIP, ufull + 8 * us);
                } else if (lane == 0) {
                    bulk_g2s(sbase + OFF_U + us * U_SLOT, w + ((int64_t)t.rt * P.chunks + kc) * Q4_UNIT_BYTES,
                             Q4_UNIT_BYTES, ufull + 8 * us);
                }
                gu++;
                // keep the weights PF stages ahead (in this item or the next one) on their way into L2
                if (kc + PF < t.nkc)
                    prefetch(t, kc + PF);
                else if (more && kc + PF - t.nkc < next.nkc)
                    prefetch(next, kc + PF - t.nkc);
                if (g >= NS && !warp_wait(empty + 8 * s, ((g / NS) - 1) & 1u)) {
                    ok = false;
                    break;
                }
                // the stage's activations: one or two 64-column boxes of `groups` x 4 rows
                const int boxes = P.K - kc * SK > KC ? 2 : 1;
                if (lane == 0) mbar_expect_tx(full_b + 8 * s, (uint32_t)(boxes * groups * 4 * KC * 2));
                __syncwarp();
                for (int b = 0; b < boxes; b++) {
                    const uint32_t dst = sbase + s * B_TILE + b * B_BOX + lane * (4 * KC * 2);
                    if (lane < groups) tma_gather4(dst, &a.bmap, kc * SK + b * KC, r[0], full_b + 8 * s);
                    if (lane + 32 < groups)
                        tma_gather4(dst + 32 * (4 * KC * 2), &a.bmap, kc * SK + b * KC, r[1], full_b + 8 * s);
                }
                __syncwarp();
            }
        }
        // Every copy this warp issued has landed before the CTA can exit, also after a wait above ran
        // out (a barrier whose phase completed long ago passes at once; a wait that runs out here ends
        // the drain).
        for (uint32_t x = g > NS ? g - NS : 0; x < g; x++)
            if (!warp_wait(full_b + 8 * (x % NS), (x / NS) & 1u)) break;
        for (uint32_t x = gu > NU ? gu - NU : 0; x < gu; x++)
            if (!warp_wait(ufull + 8 * (x % NU), (x / NU) & 1u)) break;
    } else if (warp == 1) {   // ---------------- MMA issue (one thread)
        if (lane == 0) {
            uint32_t g = 0;
            int i = 0;
            bool ok = true;
            for (int tau = blockIdx.x; tau < items && ok; tau += G, i++) {
                const Item t = item_of(a, pre, tau);
                const uint32_t idesc = mma_idesc((pairs_of(a, t).n + 15) & ~15);
                const int K = a.p[t.j].K;
                if (i >= 1 && !mbar_wait(acc_empty, (i - 1) & 1u)) break;
                tc_fence_after();
                for (int kc = 0; kc < t.nkc; kc++, g++) {
                    const uint32_t s = g % NS, par = (g / NS) & 1u;
                    if (!mbar_wait(full_a + 8 * s, par) || !mbar_wait(full_b + 8 * s, par)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = tmem + A_TMEM + s * A_COLS, bt = sbase + s * B_TILE;
                    const int steps = min(SK, K - kc * SK) / 16;   // nothing past K enters the sum
#pragma unroll
                    for (int ks = 0; ks < SK / 16; ks++)
                        if (ks < steps)
                            tc_mma(tmem, at + 8 * ks, sdesc(bt + (ks >> 2) * B_BOX + 32 * (ks & 3)), idesc,
                                   (kc | ks) != 0);
                    tc_commit(empty + 8 * s);
                }
                if (ok) tc_commit(acc_full);
            }
            tc_commit(mma_done);   // every MMA issued here is complete before the tensor memory is freed
            mbar_wait(mma_done, 0u);
        }
    } else if (warp < EPI0) {   // ---------------- warps 2..9: A conversion into tensor memory
        // lanes 32 (warp % 4) .. +31 of tensor memory are tile rows 32 (warp % 4) ..; qb: this warp
        // takes blocks qb and qb + 2 of the stage
        const int quad = warp & 3, qb = (warp - 2) >> 2, gq = lane >> 2;
        const uint32_t arow = tmem + ((uint32_t)(32 * quad) << 16) + A_TMEM;
        uint32_t g = 0;
        bool ok = true;
        for (int tau = blockIdx.x; tau < items && ok; tau += G) {
            const Item t = item_of(a, pre, tau);
            for (int kc = 0; kc < t.nkc; kc++, g++) {
                const uint32_t s = g % NS, us = g % NU;
                ok = warp_wait(ufull + 8 * us, (g / NU) & 1u);
                if (ok && g >= NS) ok = warp_wait(empty + 8 * s, ((g / NS) - 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                const uint8_t *unit = smem + OFF_U + us * U_SLOT;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int jb = 2 * h + qb;
                    const uint4 wv = load_words<WT>(unit, quad, jb, lane);
                    RowHeads<WT> hd;
                    load_heads<WT>(unit, quad, jb, gq, hd);
                    const uint4 a0 = a_word(wv.x, hd.dw[0], hd.blo[0], hd.bhi[0]);
                    const uint4 a1 = a_word(wv.y, hd.dw[1], hd.blo[1], hd.bhi[1]);
                    const uint4 a2 = a_word(wv.z, hd.dw[2], hd.blo[2], hd.bhi[2]);
                    const uint4 a3 = a_word(wv.w, hd.dw[3], hd.blo[3], hd.bhi[3]);
                    const uint32_t base = arow + s * A_COLS + 16 * jb;
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
                mbar_arrive(full_a + 8 * s);
                mbar_arrive(uempty + 8 * us);
            }
        }
    } else {   // ---------------- warps 10..25: epilogue (accumulator lane = weight row, column = pair)
        const int quad = warp & 3, c0 = ((warp - EPI0) >> 2) * 64, odd = lane & 1;
        const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)c0;
        int i = 0;
        for (int tau = blockIdx.x; tau < items; tau += G, i++) {
            const Item t = item_of(a, pre, tau);
            const IdProj &P = a.p[t.j];
            const Pairs pr = pairs_of(a, t);
            const int n = pr.n - c0;   // pairs of this column quarter
            const int id0 = lane < n ? pair_at(a, pr.first + c0 + lane) : -1;
            const int id1 = lane + 32 < n ? pair_at(a, pr.first + c0 + 32 + lane) : -1;
            if (!warp_wait(acc_full, i & 1u)) break;
            tc_fence_after();
            uint32_t h[32];
            if (n > 0) load_columns(taddr, h);
            if (n > 32) load_columns(taddr + 32u, h + 16);
            tc_fence_before();
            mbar_arrive(acc_empty);   // read: the MMAs of the next item may start
            // Rows come two at a time: lanes l and l ^ 1 exchange columns, so that the even lane holds
            // rows (l, l+1) of column 2k and the odd lane the same rows of column 2k+1: 4-byte stores.
            const int row = t.rt * TM + quad * 32 + (lane & ~1);
            const bool two = row + 1 < P.N && ((reinterpret_cast<uintptr_t>(P.y) | (uintptr_t)(P.y_stride * 2)) & 3) == 0;
            uint16_t *yr = P.y + row;
#pragma unroll
            for (int kk = 0; kk < 32; kk++) {
                if (2 * kk >= n) break;   // uniform
                const uint32_t other = __shfl_xor_sync(0xffffffffu, h[kk], 1);
                const uint32_t v = odd ? __byte_perm(other, h[kk], 0x7632) : __byte_perm(h[kk], other, 0x5410);
                const int id = __shfl_sync(0xffffffffu, kk < 16 ? id0 : id1, (2 * kk + odd) & 31);
                if (id < 0 || row >= P.N) continue;
                uint16_t *dst = yr + id * P.y_stride;
                if (two) {
                    *reinterpret_cast<uint32_t *>(dst) = v;
                } else {
                    dst[0] = (uint16_t)v;
                    if (row + 1 < P.N) dst[1] = (uint16_t)(v >> 16);
                }
            }
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
    const cudaError_t e =
        cudaFuncSetAttribute(mmq_id_kernel<WT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "mmq_id: shared memory attribute: %s", cudaGetErrorString(e));
    return launch_pdl("mmq_id", mmq_id_kernel<WT>, dim3((unsigned)sm_count()), dim3(THREADS), (size_t)SMEM_BYTES, s, a);
}

}  // namespace

int64_t mmq_id_workspace_bytes(int64_t img_rows, int64_t kmax) { return (img_rows * kmax * 2 + 127) / 128 * 128; }

qk_status read_mmq_id_faults(uint32_t *faults) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tc_faults, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_tc_faults, &zero, sizeof zero);
    if (e != cudaSuccess) return fail(QK_ERR_CUDA, "qk_device_faults: %s", cudaGetErrorString(e));
    *faults = v;
    return QK_OK;
}

qk_status launch_mmq_id(const int8_t *qs, const uint16_t *d, int64_t row_blocks, int64_t img_rows, int rows, int k,
                        int n_proj, const qk_proj_id16 *projs, const int32_t *counts, const int32_t *offsets,
                        const int32_t *items, bool per_pair, void *ws, cudaStream_t s) {
    int64_t kmax = 0;
    for (int j = 0; j < n_proj; j++) kmax = projs[j].K > kmax ? projs[j].K : kmax;
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return fail(QK_ERR_CUDA, "mmq_id: cuTensorMapEncodeTiled is not available");
    IdArgs a = {};
    const cuuint64_t dims[2] = {(cuuint64_t)kmax, (cuuint64_t)img_rows};
    const cuuint64_t strides[1] = {(cuuint64_t)kmax * 2};
    const cuuint32_t box[2] = {KC, 1}, estr[2] = {1, 1};
    const CUresult r = enc(&a.bmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, ws, dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(QK_ERR_CUDA, "mmq_id: tensor map encoding failed (%d)", (int)r);
    qk_status st = launch_dequant_b("mmq_id_dequant_b", qs, d, row_blocks, (int)img_rows, (int)kmax, ws, s);
    if (st != QK_OK) return st;
    a.counts = counts;
    a.offsets = offsets;
    a.items = items;
    a.pairs = rows * k;
    a.k = k;
    a.E = projs[0].n_experts;
    a.per_pair = per_pair;
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

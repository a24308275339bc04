// How an expert's planned pairs are cut into the passes of the routed prefill (plain C++ too, for its test).
#pragma once

#ifdef __CUDACC__
#define QK_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define QK_HOST_DEVICE inline
#endif

namespace qk {

constexpr int PASS_UNIT = 16;   // pairs; an MMA's N is a multiple of it
constexpr int PASS_MOST = 128;  // pairs of a pass at most

struct PassRange {
    int start, n;   // the pass's first pair among the expert's, and how many
};

QK_HOST_DEVICE int passes_of(int pairs) { return pairs / PASS_MOST + (pairs % PASS_MOST != 0); }

// Whole units, one more to the first passes where they do not divide: no pass is a small remainder.
QK_HOST_DEVICE PassRange pass_range(int pairs, int passes, int pass) {
    const int units = pairs / PASS_UNIT + (pairs % PASS_UNIT != 0), each = units / passes, more = units % passes;
    const int start = PASS_UNIT * (pass * each + (pass < more ? pass : more)), n = PASS_UNIT * (each + (pass < more));
    return {start, n < pairs - start ? n : pairs - start};
}

}  // namespace qk

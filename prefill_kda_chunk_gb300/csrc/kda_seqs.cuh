// Where sequences start and end, for kernels that walk a batch of them without
// a prologue launch: a block checks cu_seqlens itself, and a warp finds the
// sequence of a token with a 32-way search.
#pragma once

#include <stdint.h>

#include "kda_device.cuh"

namespace kda {

// Sequence n holds tokens [start(n), start(n + 1)): read from cu_seqlens, or n
// sequences of `len` tokens each.
struct Seqs {
    const int32_t *cu;   // [n + 1] or nullptr
    int64_t len;
    int32_t n;
    __device__ __forceinline__ int64_t start(int i) const {
        return cu != nullptr ? static_cast<int64_t>(__ldg(cu + i)) : len * i;
    }
};

// Whether cu_seqlens is 0 .. total and does not decrease (true without one).
// All threads of the block call it; block 0 records a violation. Every block
// reads the whole table once: 4 B per sequence out of L2, a pass of one load
// per thread for up to blockDim.x sequences.
__device__ __forceinline__ bool check_cu(const Seqs &s, int64_t total, int *err) {
    if (s.cu == nullptr) return true;
    int bad = 0;
    for (int i = threadIdx.x; i < s.n; i += blockDim.x) {
        const int32_t a = __ldg(s.cu + i), b = __ldg(s.cu + i + 1);
        bad |= (b < a) || (i == 0 && a != 0) || (i == s.n - 1 && b != total);
    }
    bad = __syncthreads_or(bad);
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, kErrBadCu);
    return !bad;
}

// First sequence that is not wholly before token t: the one that t continues,
// or else the first that starts at or after t (s.n if there is none). Empty
// sequences belong to the token they stand in front of. All lanes of a warp
// call it with the same t on a table that check_cu has passed.
__device__ __forceinline__ int first_seq(const Seqs &s, int64_t t) {
    if (s.cu == nullptr)
        return s.len > 0 ? static_cast<int>(t / s.len < s.n ? t / s.len : s.n) : 0;
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = s.n;   // m = number of sequences that start before t, in [lo, hi]
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + (lane + 1) * step - 1;
        const bool before = i < hi && __ldg(s.cu + i) < t;
        const int k = __popc(__ballot_sync(0xffffffffu, before));
        const int base = lo;
        lo = base + k * step;
        if (k < 32 && base + (k + 1) * step - 1 < hi) hi = base + (k + 1) * step - 1;
        if (lo > hi) lo = hi;
    }
    if (lo == 0) return 0;
    return __ldg(s.cu + lo) > t ? lo - 1 : lo;
}

}  // namespace kda

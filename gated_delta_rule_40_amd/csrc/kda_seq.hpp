// kda_seq.hpp -- device lookups in cu_seqlens for kernels over packed tokens.
// Entries are clamped to [0, T], and what is found in an array that breaks
// the rules of include/kda.h still lies in bounds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct Seqs {
    const int32_t *cu;
    int32_t N, T;
    __device__ __forceinline__ int32_t at(int32_t n) const { return min(max(cu[n], 0), T); }
    // first n in [0, N] with at(n) >= t (N + 1 if none)
    __device__ __forceinline__ int32_t first_at_or_after(int32_t t) const {
        int32_t lo = 0, hi = N + 1;
        while (lo < hi) {
            const int32_t mid = lo + (hi - lo) / 2;
            if (at(mid) >= t) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    }
    // the sequence that owns token t, or -1
    __device__ __forceinline__ int32_t owner(int32_t t) const {
        const int32_t n = first_at_or_after(t + 1) - 1;   // the last entry <= t
        return (n >= 0 && n < N) ? n : -1;
    }
};

}  // namespace kda

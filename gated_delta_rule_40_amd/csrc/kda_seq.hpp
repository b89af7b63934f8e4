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

// The same lookups for a wave around one place, from entries held a lane each:
// one read where there are at most 64 entries (it does not depend on the
// place), a few for more, against a chain of dependent reads for a binary search.
// All arguments are uniform over the wave, and all 64 lanes have to be active.
struct SeqWindow {
    Seqs sq;
    int32_t base, stride, entry;   // lane l holds entry base + l * stride

    __device__ __forceinline__ explicit SeqWindow(const Seqs &s) : sq(s), base(0), stride((s.N + 64) / 64) { read(); }
    // lanes past the last entry hold a value above every token
    __device__ __forceinline__ void read() {
        const int64_t n = base + (int64_t)(threadIdx.x & 63) * stride;
        entry = n <= sq.N ? sq.at((int32_t)n) : INT32_MAX;
    }
    __device__ __forceinline__ int below(int32_t t) const { return __popcll(__ballot(entry < t)); }
    // brings in the last entry < t and the 63 after it
    __device__ __forceinline__ void locate(int32_t t) {
        if (sq.N < 64) return;     // all are here already
        while (stride > 1) {
            const int n = below(t);
            if (n > 0) base += (n - 1) * stride;       // the last sample below t
            stride = n > 0 ? (stride + 63) / 64 : 1;   // up to the next sample
            read();
        }
        const int n = below(t);
        if (n > 1) {
            base += n - 1;
            read();
        }
    }
    __device__ __forceinline__ int32_t at(int32_t n) const {
        const int32_t i = n - base;
        return (i >= 0 && i < 64 && stride == 1) ? __builtin_amdgcn_readlane(entry, i) : sq.at(n);
    }
    // as Seqs', for t >= the place located
    __device__ __forceinline__ int32_t first_at_or_after(int32_t t) const {
        const int n = below(t);
        return n < 64 ? min(base + n, sq.N + 1) : sq.first_at_or_after(t);
    }
    __device__ __forceinline__ int32_t owner(int32_t t) const {
        const int32_t n = first_at_or_after(t + 1) - 1;
        return (n >= 0 && n < sq.N) ? n : -1;
    }
    // from sequence n, which ends before token t, to the one that begins there
    __device__ __forceinline__ void advance(int32_t t, int32_t &n, int32_t &next) const {
        if (n < sq.N - 1) next = at(++n + 1);
        if (next > t) return;
        const int32_t m = owner(t);   // past empty ones
        n = m >= 0 ? m : sq.N - 1;
        next = max(at(n + 1), t + 1);
    }
};

// Rows of states that empty sequences keep: dst[n] = src[n] (null: zeros), both
// [N][size]; a wave each, EMPTY_SEQS of them to a workgroup of its own.  They are
// found by their number, not by their place: a batch with fixed slots has
// hundreds of them at one token (511 of 512: 15 us, 320 when the wave at that
// token copied them).  Neither array may reach into the other.
constexpr int EMPTY_SEQS = 4;
template <typename T>
__device__ __forceinline__ void copy_empty(const Seqs &sq, uint32_t group, int64_t size, const T *__restrict__ src,
                                           T *__restrict__ dst)
{
    const int64_t n = (int64_t)group * EMPTY_SEQS + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (threadIdx.x >= 64 * EMPTY_SEQS || n >= sq.N || sq.at((int32_t)n + 1) > sq.at((int32_t)n)) return;
    dst += n * size;
    if (src) {
        src += n * size;
#pragma unroll 8
        for (int64_t e = threadIdx.x & 63; e < size; e += 64) dst[e] = src[e];
    } else {
        for (int64_t e = threadIdx.x & 63; e < size; e += 64) dst[e] = T(0.f);
    }
}
// workgroups that takes (none where the rows are there already)
inline int64_t empty_groups(int32_t N, const void *src, const void *dst)
{
    return dst && dst != src ? ((int64_t)N + EMPTY_SEQS - 1) / EMPTY_SEQS : 0;
}

}  // namespace kda

// kda_verify.hip -- which drafted tokens the target accepts, and the token after
// them, from given random numbers.
//
// The row of the vocabulary that the next token comes from is known once the
// accepted drafts are counted, which takes two values a draft.  So every wave counts
// them for itself, and of all rows only that one is read: its weights
// w = max(p - q, 0) are summed in parts side by side (kernel 1), and the part where
// the running sum passes sample_rand * total is searched (kernel 2; it is in the
// caches still).  Sums are formed in fp64 in a fixed order.
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_seq.hpp"

namespace kda {

constexpr int VF_THREADS = 256;
constexpr int VF_PART_MIN = 1024, VF_PART_MAX = 16384;   // weights of a part

// A sequence's verdict, the same in every lane.
struct Verdict {
    int32_t first, rows, accepted;   // first token row, token rows, drafts accepted
};

template <typename T> struct Verify {
    const T *target, *draft;
    const int32_t *tokens;
    const float *accept_rand;
    int64_t vocab;
    Seqs sq;

    // probabilities below zero and NaN count as zero
    static __device__ __forceinline__ double prob(T x) {
        const float f = to_f(x);
        return f > 0.f ? (double)f : 0.0;
    }
    // called by a whole wave
    __device__ __forceinline__ Verdict judge(int32_t n) const {
        const int32_t first = sq.at(n), rows = max(sq.at(n + 1) - first, 0), lane = threadIdx.x & 63;
        int32_t accepted = 0;
        while (accepted + 1 < rows) {
            const int32_t j = accepted + 1 + lane;   // a draft a lane
            bool good = false;
            if (j < rows) {
                const int64_t row = (int64_t)first + j;
                const int32_t x = tokens[row];
                if (x >= 0 && x < vocab) {
                    const double p = prob(target[(row - 1) * vocab + x]), q = draft ? prob(draft[row * vocab + x]) : 1.0;
                    good = (double)accept_rand[row] * q < p;
                }
            }
            const uint64_t bad = ~__ballot(good);
            const int32_t run = bad ? __builtin_ctzll(bad) : 64;
            accepted += run;
            if (run < 64) break;
        }
        return {first, rows, accepted};
    }
    // The weights of the next token's row.
    struct Row {
        const T *p, *q;     // q: the draft's row, or null
        int32_t without;    // the token that is left out (drafts picked without a distribution), or -1
        __device__ __forceinline__ double at(int32_t x) const {
            const double a = prob(p[x]);
            if (q) {
                const double d = a - prob(q[x]);
                return d > 0. ? d : 0.;
            }
            return x == without ? 0. : a;
        }
    };
    __device__ __forceinline__ Row row(const Verdict &v) const {
        const int64_t at = (int64_t)v.first + v.accepted;
        const bool rejected = v.accepted + 1 < v.rows;
        return {target + at * vocab, rejected && draft ? draft + (at + 1) * vocab : nullptr,
                rejected && !draft ? tokens[at + 1] : -1};
    }
};

// the sum over a workgroup, in every thread
__device__ __forceinline__ double group_sum(double s, double *red)
{
    for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    double t = 0.;
    for (int i = 0; i < VF_THREADS / 64; ++i) t += red[i];
    return t;
}

template <typename T>
__global__ __launch_bounds__(VF_THREADS) void kda_verify_sums_kernel(Verify<T> in, int32_t parts, int32_t part, double *sums)
{
    __shared__ double red[VF_THREADS / 64];
    const int32_t n = blockIdx.x / parts, i = blockIdx.x % parts;
    const Verdict v = in.judge(n);
    if (v.rows == 0) return;
    const auto w = in.row(v);
    const int32_t end = (int32_t)min(((int64_t)i + 1) * part, in.vocab);
    double s = 0.;
    for (int32_t x = i * part + threadIdx.x; x < end; x += VF_THREADS) s += w.at(x);
    s = group_sum(s, red);
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// The first x of [begin, end) with base + w[begin] + ... + w[x] > mark and w[x] > 0,
// or the last with w[x] > 0, or -1.
template <typename Row>
__device__ __forceinline__ int32_t search(const Row &w, int32_t begin, int32_t end, double base, double mark, double *red,
                                          int32_t *pick)
{
    const int32_t per = (end - begin + VF_THREADS - 1) / VF_THREADS;
    const int32_t mine = min(begin + (int32_t)threadIdx.x * per, end), stop = min(mine + per, end);
    double s = 0.;
    for (int32_t x = mine; x < stop; ++x) s += w.at(x);
    // sums of the threads before this one
    double before = s;
    for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_up(before, off);
        if ((int)(threadIdx.x & 63) >= off) before += y;
    }
    __syncthreads();   // (a sum may have been read from `red` just now)
    if ((threadIdx.x & 63) == 63) red[threadIdx.x >> 6] = before;
    if (threadIdx.x == 0) pick[0] = INT32_MAX, pick[1] = -1;
    __syncthreads();
    before -= s;
    for (int i = 0; i < (int)(threadIdx.x >> 6); ++i) before += red[i];
    double sum = base + before;
    int32_t found = INT32_MAX, last = -1;
    for (int32_t x = mine; x < stop; ++x) {
        const double y = w.at(x);
        sum += y;
        if (y > 0.) {
            last = x;
            if (found == INT32_MAX && sum > mark) found = x;
        }
    }
    if (found != INT32_MAX) atomicMin(&pick[0], found);
    if (last >= 0) atomicMax(&pick[1], last);
    __syncthreads();
    return pick[0] != INT32_MAX ? pick[0] : pick[1];
}

template <typename T>
__global__ __launch_bounds__(VF_THREADS) void kda_verify_pick_kernel(Verify<T> in, const float *sample_rand, int32_t parts,
                                                                     int32_t part, const double *sums, int32_t *num_tokens,
                                                                     int32_t *next_token)
{
    __shared__ double red[VF_THREADS / 64];
    __shared__ int32_t pick[2];
    const int32_t n = blockIdx.x;
    const Verdict v = in.judge(n);
    if (v.rows == 0) {
        if (threadIdx.x == 0) num_tokens[n] = 0, next_token[n] = -1;
        return;
    }
    auto w = in.row(v);
    sums += (int64_t)n * parts;
    double total = 0.;
    for (int32_t i = 0; i < parts; ++i) total += sums[i];
    int32_t begin = 0, end = (int32_t)in.vocab;
    double base = 0.;
    if (total == 0. && (w.q || w.without >= 0)) {   // nothing is left: the target's own row, whole
        w.q = nullptr, w.without = -1;
        double s = 0.;
        for (int32_t x = threadIdx.x; x < in.vocab; x += VF_THREADS) s += w.at(x);
        total = group_sum(s, red);
    } else {
        // the part in which the running sum passes the mark, or the last that has a weight
        int32_t at = 0;
        double sum = 0.;
        for (int32_t i = 0; i < parts; ++i) {
            if (!(sums[i] > 0.)) continue;
            at = i, base = sum;
            sum += sums[i];
            if (sum > (double)sample_rand[n] * total) break;
        }
        begin = at * part;
        end = (int32_t)min((int64_t)begin + part, in.vocab);
    }
    const int32_t x = search(w, begin, end, base, (double)sample_rand[n] * total, red, pick);
    if (threadIdx.x == 0) num_tokens[n] = 1 + v.accepted, next_token[n] = x;
}

// weights of a part: about 2,048 workgroups in all
inline int32_t part_size(int32_t N, int32_t vocab)
{
    int64_t part = (int64_t)vocab * N / 2048;
    part = part < VF_PART_MIN ? VF_PART_MIN : part > VF_PART_MAX ? VF_PART_MAX : part;
    return (int32_t)((part + VF_THREADS - 1) / VF_THREADS * VF_THREADS);
}
inline int32_t part_count(int32_t N, int32_t vocab)
{
    const int32_t part = part_size(N, vocab);
    return (int32_t)(((int64_t)vocab + part - 1) / part);
}

}  // namespace kda

using namespace kda;

size_t kda_verify_ws_bytes(int32_t N, int32_t vocab) { return (size_t)N * part_count(N, vocab) * sizeof(double); }

bool kda_verify_fits(int32_t N, int32_t vocab)
{
    return (int64_t)N * part_count(N, vocab) <= INT32_MAX && kda_grid_ok((int64_t)N * part_count(N, vocab), VF_THREADS);
}

template <typename T>
static hipError_t verify(const void *target, const void *draft, const int32_t *tokens, const int32_t *cu,
                         const float *accept_rand, const float *sample_rand, int32_t N, int32_t T_tot, int32_t vocab,
                         int32_t *num_tokens, int32_t *next_token, void *ws, hipStream_t s)
{
    const Verify<T> in{(const T *)target, (const T *)draft, tokens, accept_rand, vocab, {cu, N, T_tot}};
    const int32_t part = part_size(N, vocab), parts = part_count(N, vocab);
    hipLaunchKernelGGL(kda_verify_sums_kernel<T>, dim3((unsigned)(N * parts)), dim3(VF_THREADS), 0, s, in, parts, part,
                       (double *)ws);
    hipLaunchKernelGGL(kda_verify_pick_kernel<T>, dim3((unsigned)N), dim3(VF_THREADS), 0, s, in, sample_rand, parts, part,
                       (const double *)ws, num_tokens, next_token);
    return hipGetLastError();
}

hipError_t kda_launch_verify(bool bf16, const void *target, const void *draft, const int32_t *tokens, const int32_t *cu,
                             const float *accept_rand, const float *sample_rand, int32_t N, int32_t T_tot, int32_t vocab,
                             int32_t *num_tokens, int32_t *next_token, void *ws, hipStream_t s)
{
    return bf16 ? verify<bf16_t>(target, draft, tokens, cu, accept_rand, sample_rand, N, T_tot, vocab, num_tokens, next_token,
                                 ws, s)
                : verify<float>(target, draft, tokens, cu, accept_rand, sample_rand, N, T_tot, vocab, num_tokens, next_token,
                                ws, s);
}

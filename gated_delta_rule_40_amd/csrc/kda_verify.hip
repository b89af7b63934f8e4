// kda_verify.hip -- which drafted tokens the target accepts, and the token after
// them, from given random numbers.
//
// The row of the vocabulary that the next token comes from is known once the
// accepted drafts are counted, which takes two values a draft.  So every workgroup
// counts them for itself, and of all rows only that one is read: its weights
// w = max(p - q, 0) are summed in parts of 1,024, a wave each (kernel 1), and the part
// where the running sum passes sample_rand * total is searched (kernel 2).
//
// Sums are formed in fp64 in a fixed order.  A difference has its sign exactly and is
// rounded once (fp32 probabilities may lie more than 53 binary places apart).  No
// partial sum is above the total, so every rounding is off by at most u = 2^-53 of it.
// With P = ceil(vocab / 2^18) parts a thread, the total passes at most 36 + P roundings
// (1 of the difference, 8 in a lane, 6 over lanes, P, 6 over lanes, 15 over waves), the
// mark one more, and the running sum at a place 69 + 2 P (36 + 2 P + 1 up to its part, 32
// within).  So a token is the one that real numbers give unless the mark lies within
// (106 + 3 P) u of the total from a running sum: 2^-46 up to 2^18 tokens, 2^-39 at 2^30.
// (Where nothing is left and the target's row is summed by one workgroup, each thread
// adds 1,024 P weights and 256 P parts: (110 + 1,300 P) u, 2^-42 and 2^-30.)
//
// HBM bounds large calls, latency small ones: the counting takes two dependent reads,
// each kernel about three.  One MI355X, fp32, four drafts, both kernels of a replayed
// graph: 256 sequences of 131,072 42 us (kernel 1 37, 5.8 TB/s), 256 x 32,000 16 us, one
// of 32,000 6.3 us.  Read through the caches, rows take 10-20 % longer.  Small rows of few
// sequences are done in one launch.
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_seq.hpp"

#include <type_traits>

namespace kda {

constexpr int VF_THREADS = 256, VF_WAVES = VF_THREADS / 64;
constexpr int VF_PART = 1024;   // weights that one wave sums, and that are searched at once

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
    static __device__ __forceinline__ double prob(T x) { return (double)fmaxf(to_f(x), 0.f); }
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
        int32_t vocab;

        // VW consecutive weights from x0 on, zeros beyond the row; q's part is read with p's
        template <int VW> __device__ __forceinline__ void read(int32_t x0, T (&a)[VW], T (&b)[VW]) const {
            typedef T raw __attribute__((ext_vector_type(VW)));
            typedef raw mem __attribute__((aligned(sizeof(T))));
            raw u{}, v{};
            if (x0 + VW <= vocab) {
                u = __builtin_nontemporal_load(reinterpret_cast<const mem *>(p + x0));
                if (q) v = __builtin_nontemporal_load(reinterpret_cast<const mem *>(q + x0));
            } else {
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    if (x0 + j < vocab) {
                        u[j] = p[x0 + j];
                        if (q) v[j] = q[x0 + j];
                    }
            }
#pragma unroll
            for (int j = 0; j < VW; ++j) a[j] = u[j], b[j] = v[j];
        }
        __device__ __forceinline__ double weight(int32_t x, T a, T b) const {
            const double w = fmax(prob(a) - prob(b), 0.);   // (infinity less infinity: zero)
            return x == without ? 0. : w;
        }
    };
    __device__ __forceinline__ Row row(const Verdict &v) const {
        const int64_t at = (int64_t)v.first + v.accepted;
        const bool rejected = v.accepted + 1 < v.rows;
        return {target + at * vocab, rejected && draft ? draft + (at + 1) * vocab : nullptr,
                rejected && !draft ? tokens[at + 1] : -1, (int32_t)vocab};
    }
};

// The sums up to each lane of a wave: within rows of 16 lanes, then over the rows.
template <int CTRL, int ROWS> __device__ __forceinline__ double add_from(double x)
{
    union { double d; int i[2]; } u{x}, y;
    y.i[0] = __builtin_amdgcn_update_dpp(0, u.i[0], CTRL, ROWS, 0xf, true);
    y.i[1] = __builtin_amdgcn_update_dpp(0, u.i[1], CTRL, ROWS, 0xf, true);
    return x + y.d;   // (lanes without a source add zero)
}
__device__ __forceinline__ double wave_scan(double s)
{
    s = add_from<0x111, 0xf>(s);   // row_shr:1
    s = add_from<0x112, 0xf>(s);
    s = add_from<0x114, 0xf>(s);
    s = add_from<0x118, 0xf>(s);
    s = add_from<0x142, 0xa>(s);   // row_bcast:15 into rows 1 and 3
    return add_from<0x143, 0xc>(s);   // row_bcast:31 into rows 2 and 3
}

// The sums of parts `part` to part + K - 1 of a row, by one wave, in its last lane.
template <typename T, int K> __device__ __forceinline__ void part_sums(const typename Verify<T>::Row &w, int32_t part, double (&sum)[K])
{
    constexpr int VW = 16 / sizeof(T), PIECES = VF_PART / 64 / VW;
    const int32_t x0 = part * VF_PART + (threadIdx.x & 63) * VW;
    T a[K * PIECES][VW], b[K * PIECES][VW];
#pragma unroll
    for (int c = 0; c < K * PIECES; ++c) w.template read<VW>(x0 + c * 64 * VW, a[c], b[c]);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        sum[k] = 0.;
#pragma unroll
        for (int c = k * PIECES; c < (k + 1) * PIECES; ++c) {
            double s = 0.;
#pragma unroll
            for (int j = 0; j < VW; ++j) s += w.weight(x0 + c * 64 * VW + j, a[c][j], b[c][j]);
            sum[k] += s;
        }
        sum[k] = wave_scan(sum[k]);
    }
}

// What a workgroup finds: every thread has the weights of some places, `run` their
// sum, in the order of the threads.
template <int THREADS> struct Search {
    static constexpr int WAVES = THREADS / 64;
    double waves[WAVES];
    double base;                                // the sum before the part that is searched
    int32_t firsts[WAVES], lasts[WAVES];

    // The sum before this thread's places, and of all (called by the whole workgroup).
    __device__ __forceinline__ double before(double run, double &total) {
        const double s = wave_scan(run);
        __syncthreads();   // (the search before is over)
        if ((threadIdx.x & 63) == 63) waves[threadIdx.x >> 6] = s;
        __syncthreads();
        double up = s - run;
        total = 0.;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            if (i == (int)(threadIdx.x >> 6)) up += total;
            total += waves[i];
        }
        return up;
    }
    // From every thread's first place that passes the mark (INT32_MAX: none) and last
    // that has a weight (-1), those of all: places go up with the threads, so they are
    // the lowest lane's and the highest lane's.  (Atomics on two words of LDS, 256
    // threads each, took 2 to 4 us.)
    __device__ __forceinline__ void found(int32_t &first, int32_t &last) {
        const uint64_t passed = __ballot(first != INT32_MAX), some = __ballot(last >= 0);
        const int32_t f = __shfl(first, passed ? __builtin_ctzll(passed) : 0);
        const int32_t l = __shfl(last, some ? 63 - __builtin_clzll(some) : 0);
        if ((threadIdx.x & 63) == 0) firsts[threadIdx.x >> 6] = f, lasts[threadIdx.x >> 6] = l;
        __syncthreads();
        first = INT32_MAX, last = -1;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) first = min(first, firsts[i]), last = max(last, lasts[i]);
    }

    // The next token, given the sums of the row's parts.  The first place x with
    // w[x] > 0 whose running sum is above the mark lies in the first part with a
    // weight whose running sum is (running sums of weights never fall); if there is
    // none, the last place with a weight in the last such part.
    // A thread has parts [p0, p1), whose sum is `run`.
    template <typename T>
    __device__ __forceinline__ int32_t pick(typename Verify<T>::Row w, const double *sums, int32_t parts, int32_t p0, int32_t p1,
                                            double run, double sample) {
        constexpr int VW = VF_PART / THREADS;
        double total, sum = before(run, total);
        const bool whole = total == 0. && (w.q || w.without >= 0);   // nothing is left: the target's own row
        if (whole) {
            w.q = nullptr, w.without = -1;
            run = 0.;
            for (int32_t x0 = threadIdx.x * VW; x0 < w.vocab; x0 += VF_PART) {
                T a[VW], b[VW];
                w.template read<VW>(x0, a, b);
#pragma unroll
                for (int j = 0; j < VW; ++j) run += w.weight(x0 + j, a[j], b[j]);
            }
            before(run, total);
        }
        const double mark = sample * total;
        int32_t part = 0, end = parts;
        double from = 0.;
        if (!whole) {
            int32_t mine_first = INT32_MAX, mine_last = -1;
            double first_base = 0., last_base = 0.;
            for (int32_t i = p0; i < p1; ++i) {
                const double s = sums[i];
                if (s > 0.) {
                    mine_last = i, last_base = sum;
                    if (mine_first == INT32_MAX && sum + s > mark) mine_first = i, first_base = sum;
                }
                sum += s;
            }
            int32_t first = mine_first, last = mine_last;
            found(first, last);
            part = max(first != INT32_MAX ? first : last, 0);
            if (part >= p0 && part < p1) base = part == mine_first ? first_base : last_base;
            end = part + 1;
            __syncthreads();
            from = base;
        }
        // the part; of a whole row the parts in turn, to the first that has it
        int32_t next = -1;
        for (; part < end; ++part) {
            const int32_t x0 = part * VF_PART + threadIdx.x * VW;
            T a[VW], b[VW];
            double y[VW];
            w.template read<VW>(x0, a, b);
            run = 0.;
#pragma unroll
            for (int j = 0; j < VW; ++j) y[j] = w.weight(x0 + j, a[j], b[j]), run += y[j];
            double all;
            sum = from + before(run, all);
            int32_t first = INT32_MAX, last = -1;
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                sum += y[j];
                if (y[j] > 0.) {
                    last = x0 + j;
                    if (first == INT32_MAX && sum > mark) first = x0 + j;
                }
            }
            found(first, last);
            next = first != INT32_MAX ? first : max(next, last);
            if (first != INT32_MAX) break;
            from += all;
        }
        return next;
    }
};

// Kernel 1: a row's parts over many workgroups.  A wave takes K of them, all reads
// before the first use.
template <typename T, int K>
__global__ __launch_bounds__(VF_THREADS) void kda_verify_sums_kernel(Verify<T> in, int32_t groups, int32_t parts, double *sums,
                                                                     int32_t *counts)
{
    const int32_t n = blockIdx.x / groups, group = blockIdx.x % groups;
    const int32_t part = (group * VF_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * K;
    const Verdict v = in.judge(n);
    if (group == 0 && threadIdx.x == 0) counts[n] = v.accepted;
    if (v.rows == 0 || part >= parts) return;
    double s[K];
    part_sums<T, K>(in.row(v), part, s);
    if ((threadIdx.x & 63) == 63)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (part + k < parts) sums[(int64_t)n * parts + part + k] = s[k];
}

// Kernel 2: a workgroup a sequence.
template <typename T>
__global__ __launch_bounds__(VF_THREADS) void kda_verify_pick_kernel(Verify<T> in, const float *sample_rand, int32_t parts,
                                                                     const double *sums, const int32_t *counts,
                                                                     int32_t *num_tokens, int32_t *next_token)
{
    __shared__ Search<VF_THREADS> find;
    const int32_t n = blockIdx.x;
    const Verdict v{in.sq.at(n), max(in.sq.at(n + 1) - in.sq.at(n), 0), counts[n]};
    const double sample = sample_rand[n];
    sums += (int64_t)n * parts;
    const int32_t per = (parts + VF_THREADS - 1) / VF_THREADS;
    const int32_t p0 = min((int32_t)threadIdx.x * per, parts), p1 = min(p0 + per, parts);
    double run = 0.;
    for (int32_t i = p0; i < p1; ++i) run += sums[i];
    asm volatile("" ::: "memory");   // (keeps these reads ahead of what waits for the counts)
    if (v.rows == 0) {
        if (threadIdx.x == 0) num_tokens[n] = 0, next_token[n] = -1;
        return;
    }
    const int32_t next = find.template pick<T>(in.row(v), sums, parts, p0, p1, run, sample);
    if (threadIdx.x == 0) num_tokens[n] = 1 + v.accepted, next_token[n] = next;
}

// Both in one launch: a workgroup of 16 waves a sequence, a part a wave, sums in LDS.
constexpr int VF_ONE_THREADS = 1024, VF_ONE_PARTS = 16;
template <typename T>
__global__ __launch_bounds__(VF_ONE_THREADS) void kda_verify_one_kernel(Verify<T> in, const float *sample_rand, int32_t parts,
                                                                        int32_t *num_tokens, int32_t *next_token)
{
    __shared__ Search<VF_ONE_THREADS> find;
    __shared__ double sums[VF_ONE_PARTS];
    const int32_t n = blockIdx.x, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const double sample = sample_rand[n];
    const Verdict v = in.judge(n);
    if (v.rows == 0) {
        if (threadIdx.x == 0) num_tokens[n] = 0, next_token[n] = -1;
        return;
    }
    const auto row = in.row(v);
    if (wave < parts) {   // (at most as many as waves)
        double s[1];
        part_sums<T, 1>(row, wave, s);
        if ((threadIdx.x & 63) == 63) sums[wave] = s[0];
    }
    __syncthreads();
    const int32_t p0 = min((int32_t)threadIdx.x, parts), p1 = min(p0 + 1, parts);
    const int32_t next = find.template pick<T>(row, sums, parts, p0, p1, p0 < p1 ? sums[p0] : 0., sample);
    if (threadIdx.x == 0) num_tokens[n] = 1 + v.accepted, next_token[n] = next;
}

inline int32_t part_count(int32_t vocab) { return (int32_t)(((int64_t)vocab + VF_PART - 1) / VF_PART); }
// One launch for rows of up to 16 parts and as many sequences as CUs: a call's time is the
// host's, 8.2 us for 10.9 (fp32, one, 16 or 61 of 8,000); replayed one of 8,000 takes 6.5 us for
// 6.3, 256 8.8 for 8.8, one of 16,000 7.8 for 6.2, 256 10.7 for 11.5.  Above, one CU reads a row too
// slowly (one of 32,000 9.7 for 6.3), or two workgroups share one (512 of 8,000 16.5 for 12.0).
inline bool one_launch(int32_t N, int32_t parts) { return parts <= VF_ONE_PARTS && N <= 256; }
// Parts of a wave: two from 16,384 parts on (us of both kernels, one and two: 256 rows of
// 131,072 46.3 and 42.4, 400 of 65,537 39.4 and 37.2, 128 of 131,072 26.7 and 25.7; 64 of
// 131,072 15.8 and 16.4, one of 32,000 6.1 and 7.0).
inline int parts_each(int32_t N, int32_t vocab)
{
    return N * (int64_t)part_count(vocab) < 16384 ? 1 : 2;
}
// workgroups of a sequence
inline int64_t sum_groups(int32_t N, int32_t vocab)
{
    const int64_t per = VF_WAVES * (int64_t)parts_each(N, vocab);
    return (part_count(vocab) + per - 1) / per;
}

}  // namespace kda

using namespace kda;

// the parts' sums, and the drafts accepted
size_t kda_verify_ws_bytes(int32_t N, int32_t vocab)
{
    return (size_t)N * part_count(vocab) * sizeof(double) + (size_t)N * sizeof(int32_t);
}

bool kda_verify_fits(int32_t N, int32_t vocab) { return kda_grid_ok(N * sum_groups(N, vocab), VF_THREADS); }

template <typename T>
static hipError_t verify(const void *target, const void *draft, const int32_t *tokens, const int32_t *cu,
                         const float *accept_rand, const float *sample_rand, int32_t N, int32_t T_tot, int32_t vocab,
                         int32_t *num_tokens, int32_t *next_token, void *ws, hipStream_t s)
{
    const Verify<T> in{(const T *)target, (const T *)draft, tokens, accept_rand, vocab, {cu, N, T_tot}};
    const int32_t parts = part_count(vocab), groups = (int32_t)sum_groups(N, vocab);
    double *const sums = (double *)ws;
    int32_t *const counts = (int32_t *)(sums + (size_t)N * parts);
    if (one_launch(N, parts)) {
        hipLaunchKernelGGL(kda_verify_one_kernel<T>, dim3((unsigned)N), dim3(VF_ONE_THREADS), 0, s, in, sample_rand, parts,
                           num_tokens, next_token);
        return hipGetLastError();
    }
    const auto sum = [&](auto k) {
        hipLaunchKernelGGL((kda_verify_sums_kernel<T, k()>), dim3((unsigned)(N * (int64_t)groups)), dim3(VF_THREADS), 0, s, in,
                           groups, parts, sums, counts);
    };
    if (parts_each(N, vocab) == 1) sum(std::integral_constant<int, 1>());
    else sum(std::integral_constant<int, 2>());
    hipLaunchKernelGGL(kda_verify_pick_kernel<T>, dim3((unsigned)N), dim3(VF_THREADS), 0, s, in, sample_rand, parts, sums,
                       counts, num_tokens, next_token);
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

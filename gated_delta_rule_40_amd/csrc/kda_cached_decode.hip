// kda_cached_decode.hip -- a few tokens per (sequence, head) on states that stay in
// a cache in 8 or 4 bits.
//
// Per token, as in kda_decode.hip: Sbar = Diag(exp(g)) S, a = Sbar^T k, b = Sbar^T q,
// u = v - a, S' = Sbar + beta k u^T, o = b + beta (q.k) u.  The state is read from
// its codes, kept in fp32 registers over the tokens, and rounded once when it is
// written back, each block of 32 columns of a row with a scale of its own.
//
// The columns of a state do not depend on each other, so a wave takes one block of
// 32 columns of all 128 rows: nothing is exchanged between waves, and there is no
// barrier.  A lane holds 16 columns of four rows (two lanes a row); sums over the
// rows are formed by halving: every exchange with a lane leaves each of the two
// with half of the sums, until a lane has one column of a or b.
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_mx.hpp"

namespace kda {

constexpr int CD = 128;                       // dk = dv
constexpr int CD_WAVES = CD / MXB;            // waves of a (sequence, head): its blocks of columns
constexpr int CD_THREADS = 64 * CD_WAVES;
constexpr int CD_ROWS = 4;                    // rows of a lane: lane / 2 + 32 i
constexpr int CD_COLS = 16;                   // columns of a lane

// x[i] += x[i + M] of this lane and its partner's, halving the sums a lane holds.
template <int M> __device__ __forceinline__ void halve32(float *x)
{
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[i]), __float_as_uint(x[i + M]), false, false);
        x[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
}
template <int M> __device__ __forceinline__ void halve16(float *x)
{
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[i]), __float_as_uint(x[i + M]), false, false);
        x[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
}
template <int M, typename Fn> __device__ __forceinline__ void halve(float *x, bool upper, Fn from_partner)
{
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const float keep = upper ? x[i + M] : x[i], send = upper ? x[i] : x[i + M];
        x[i] = keep + from_partner(send);
    }
}

template <typename T, typename F>
__global__ __launch_bounds__(CD_THREADS) void kda_cached_tokens_kernel(
    const T *q, const T *k, const T *v, const float *g, const float *beta, const int32_t *cu, const int32_t *num_tokens,
    uint8_t *cache, uint8_t *scales, const int32_t *slots, int32_t write, int32_t num_slots, int32_t H, int32_t T_tot,
    int64_t units, T *out)
{
    constexpr int WORDS = CD_COLS * F::BITS / 32;   // of a lane's codes in a row
    typedef uint32_t words __attribute__((ext_vector_type(WORDS)));
    typedef words words_mem __attribute__((aligned(1)));
    __shared__ float su[CD_WAVES][MXB];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane & 1, r0 = lane >> 1;
    const int64_t u = blockIdx.x;
    const int32_t n = (int32_t)(u / H), h = (int32_t)(u % H);
    const int32_t t0 = min(max(cu[n], 0), T_tot);
    int32_t len = min(max(cu[n + 1], t0), T_tot) - t0;
    if (num_tokens) len = min(len, max(num_tokens[n], 0));
    if (len == 0) return;
    const int32_t slot = slots[n];
    const bool kept = slot >= 0 && slot < num_slots;
    const int64_t entry = ((int64_t)slot * H + h) * CD;   // rows before this state's

    float s[CD_ROWS][CD_COLS];
#pragma unroll
    for (int i = 0; i < CD_ROWS; ++i) {
        const int64_t row = entry + r0 + 32 * i;
        words w = {};
        int sc = 127;
        if (kept) {
            w = *reinterpret_cast<const words_mem *>(cache + (row * CD + wave * MXB + half * CD_COLS) * F::BITS / 8);
            sc = scales[row * CD_WAVES + wave];
        }
        const float down = mx_down<F>(sc);
#pragma unroll
        for (int j = 0; j < CD_COLS; j += 32 / F::BITS) F::decode(w[j * F::BITS / 32], &s[i][j]);
#pragma unroll
        for (int j = 0; j < CD_COLS; ++j) s[i][j] *= down;
    }

    // the column whose sums this lane has after the halving (lanes of the lower half: a, of the upper: b)
    const int col = half * CD_COLS + ((lane >> 1 & 8) | (lane >> 1 & 4) | (lane >> 1 & 2) | (lane >> 1 & 1));
    for (int32_t t = 0; t < len; ++t) {
        const int64_t row = (int64_t)(t0 + t) * H + h;
        float kk[CD_ROWS], x[2 * CD_COLS] = {}, qk = 0.f;
#pragma unroll
        for (int i = 0; i < CD_ROWS; ++i) {
            const int64_t at = row * CD + r0 + 32 * i;
            kk[i] = to_f(k[at]);
            const float qq = to_f(q[at]), decay = expf(g[at]);
            qk += kk[i] * qq;
#pragma unroll
            for (int j = 0; j < CD_COLS; ++j) {
                s[i][j] *= decay;
                x[j] += s[i][j] * kk[i];
                x[CD_COLS + j] += s[i][j] * qq;
            }
        }
#pragma unroll
        for (int off = 2; off < 64; off <<= 1) qk += __shfl_xor(qk, off);
        halve32<16>(x);
        halve16<8>(x);
        halve<4>(x, lane & 8, [](float y) { return dpp<DPP_ROR8>(y); });
        halve<2>(x, lane & 4, [](float y) { return __shfl_xor(y, 4); });
        halve<1>(x, lane & 2, [](float y) { return dpp<DPP_XOR2>(y); });
        const float b = __shfl_xor(x[0], 32), bt = beta[row];
        if (lane < 32) {
            const int64_t at = row * CD + wave * MXB + col;
            const float off = bt * (to_f(v[at]) - x[0]);
            su[wave][col] = off;
            if (out) out[at] = from_f<T>(b + qk * off);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float off[CD_COLS];
#pragma unroll
        for (int j = 0; j < CD_COLS; ++j) off[j] = su[wave][half * CD_COLS + j];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < CD_ROWS; ++i)
#pragma unroll
            for (int j = 0; j < CD_COLS; ++j) s[i][j] += kk[i] * off[j];
    }
    if (!write || !kept) return;
#pragma unroll
    for (int i = 0; i < CD_ROWS; ++i) {
        const int64_t row = entry + r0 + 32 * i;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < CD_COLS; ++j) top = max(top, __float_as_uint(s[i][j]) & 0x7fffffffu);
        top = max(top, dpp<DPP_XOR1>(top));
        const int sc = mx_scale_of<F>(top);
        const float up = mx_up(sc);
        words w;
#pragma unroll
        for (int j = 0; j < WORDS; ++j) w[j] = sc == 255 ? 0 : F::encode(&s[i][j * 32 / F::BITS], up);
        *reinterpret_cast<words_mem *>(cache + (row * CD + wave * MXB + half * CD_COLS) * F::BITS / 8) = w;
        if (half == 0) scales[row * CD_WAVES + wave] = (uint8_t)sc;
    }
}

}  // namespace kda

using namespace kda;

template <typename T>
static hipError_t cached_tokens(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                const int32_t *cu, const int32_t *num_tokens, uint8_t *cache, uint8_t *scales,
                                const int32_t *slots, bool write, int32_t num_slots, int32_t N, int32_t T_tot, int32_t H,
                                int format, void *out, hipStream_t s)
{
    return with_format(format, [&](auto f) {
        hipLaunchKernelGGL((kda_cached_tokens_kernel<T, decltype(f)>), dim3((unsigned)((int64_t)N * H)), dim3(CD_THREADS), 0, s,
                           (const T *)q, (const T *)k, (const T *)v, g, beta, cu, num_tokens, cache, scales, slots,
                           (int32_t)write, num_slots, H, T_tot, (int64_t)N * H, (T *)out);
        return hipGetLastError();
    });
}

bool kda_cached_tokens_fits(int32_t N, int32_t H) { return kda_grid_ok((int64_t)N * H, CD_THREADS); }

hipError_t kda_launch_cached_tokens(bool bf16, const void *q, const void *k, const void *v, const float *g, const float *beta,
                                    const int32_t *cu, const int32_t *num_tokens, uint8_t *cache, uint8_t *scales,
                                    const int32_t *slots, bool write, int32_t num_slots, int32_t N, int32_t T_tot,
                                    int32_t H, int format, void *out, hipStream_t s)
{
    return bf16 ? cached_tokens<bf16_t>(q, k, v, g, beta, cu, num_tokens, cache, scales, slots, write, num_slots, N, T_tot, H,
                                        format, out, s)
                : cached_tokens<float>(q, k, v, g, beta, cu, num_tokens, cache, scales, slots, write, num_slots, N, T_tot, H,
                                       format, out, s);
}

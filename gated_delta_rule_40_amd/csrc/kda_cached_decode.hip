// kda_cached_decode.hip -- a few tokens per (sequence, head) on states that stay in
// a cache in 8 or 4 bits.
//
// Per token, as in kda_decode.hip: Sbar = Diag(exp(g)) S, a = Sbar^T k, b = Sbar^T q,
// u = v - a, S' = Sbar + beta k u^T, o = b + beta (q.k) u.  The state is read from
// its codes, kept in fp32 registers over the tokens, and rounded once when it is
// written back, each block of 32 columns of a row with a scale of its own.
//
// A workgroup of four waves takes a (sequence, head).  A wave has 32 rows, a lane 16
// columns of four of them, so that a read or write of the wave is 1 KB in a row.
// The sums over the rows of a wave are formed by halving: every exchange with a lane
// leaves each of the two with half of the sums.  Those of the four waves meet in LDS,
// which takes one barrier a token: every wave adds them up for itself.
//
// HBM bounds one token (33 KB of codes and scales a state, past the caches), vector
// instructions several (about 380 a wave and token for 64 values a lane: the decay, two
// products, the update, and the halving).  One MI355X, bf16, replays of a graph: 512
// sequences of 32 heads, one token committed, fp8 104-106 us (5.5 TB/s), int8 106, fp4 88;
// five tokens verified 213, committed without outputs 131; 8 x 8 heads 4.5.
// Waves that each had 32 columns of all rows needed no barrier, but their reads of 32
// bytes a row bound them to 129 us; 8 columns by 8 rows a lane 119 (198 for five tokens
// verified); decays kept apart from the state, as factors of its rows, gained 4 % for
// five tokens and lost 1-4 % for one.
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_mx.hpp"

namespace kda {

constexpr int CD = 128;                       // dk = dv
constexpr int CD_WAVES = 4, CD_THREADS = 64 * CD_WAVES;
constexpr int CD_BLOCKS = CD / MXB;           // blocks of a row
constexpr int CD_COLS = 16;                   // columns of a lane: 16 (lane % 8) on
constexpr int CD_LANES = CD / CD_COLS;        // lanes of a row
constexpr int CD_APART = 64 / CD_LANES;       // rows of a lane: lane / 8 + 8 i, of its wave's 32
constexpr int CD_ROWS = 4, CD_WROWS = CD / CD_WAVES;

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

// the sum over each half of a wave, in every lane
__device__ __forceinline__ float sum_half_wave(float x)
{
    x += dpp<DPP_XOR1>(x);
    x += dpp<DPP_XOR2>(x);
    x += dpp<DPP_HALF_MIRROR>(x);
    x += dpp<DPP_MIRROR>(x);
    return add_xor16(x);
}

// What a lane reads of a token: key, query and gate of one of its wave's rows (lanes
// 32 on: again), two values, and beta.
template <typename T> struct Token {
    typedef T two __attribute__((ext_vector_type(2)));
    T k, q;
    two v;
    float g, beta;
};

// OUT: with outputs (else a and the states alone).
template <typename T, typename F, bool OUT>
__global__ __launch_bounds__(CD_THREADS, 3) void kda_cached_tokens_kernel(
    const T *q, const T *k, const T *v, const float *g, const float *beta, const int32_t *cu, const int32_t *num_tokens,
    uint8_t *cache, uint8_t *scales, const int32_t *slots, int32_t write, int32_t num_slots, int32_t H,
    uint32_t per_head, int32_t shift, int32_t T_tot, T *out)
{
    constexpr int WORDS = CD_COLS * F::BITS / 32;   // of a lane's codes in a row
    constexpr int ROW_BYTES = CD * F::BITS / 8;
    typedef uint32_t words __attribute__((ext_vector_type(WORDS)));
    typedef words words_mem __attribute__((aligned(1)));
    typedef uint32_t word_mem __attribute__((aligned(1)));
    typedef typename Token<T>::two two_mem __attribute__((aligned(sizeof(T))));
    __shared__ f32x4 rows[CD_WAVES][CD_WROWS];                  // key, query, decay (and at first the scale bytes)
    __shared__ float sums[2][CD_WAVES][2][CD], dots[2][CD_WAVES];   // of the waves: a and b; q.k
    __shared__ float offs[CD_WAVES][CD];                        // a wave's own copy of beta u

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int side = lane % CD_LANES, r0 = lane / CD_LANES;
    const uint32_t u = blockIdx.x;
    const int32_t n = (int32_t)((uint64_t)u * per_head >> shift), h = (int32_t)u - n * H;   // u / H, u % H
    const int32_t t0 = min(max(cu[n], 0), T_tot);
    int32_t len = min(max(cu[n + 1], t0), T_tot) - t0;
    if (num_tokens) len = min(len, max(num_tokens[n], 0));
    const int32_t slot = slots[n];
    if (len == 0) return;

    const int my_row = lane % CD_WROWS;
    const auto read = [&](int32_t t) {
        const int64_t row = ((int64_t)(t0 + t) * H + h) * CD, at = row + wave * CD_WROWS + my_row;
        Token<T> x{};
        x.k = k[at], x.g = g[at];
        if (OUT) x.q = q[at];
        x.v = *reinterpret_cast<const two_mem *>(v + row + 2 * lane);
        x.beta = beta[(int64_t)(t0 + t) * H + h];
        return x;
    };
    const bool kept = slot >= 0 && slot < num_slots;
    const int64_t entry = (((int64_t)slot * H + h) * CD) + wave * CD_WROWS;   // rows before this wave's
    uint8_t *const codes = cache + (entry + r0) * ROW_BYTES + side * (CD_COLS * F::BITS / 8);
    words w[CD_ROWS];
    uint32_t sc = 0x7f7f7f7f;
#pragma unroll
    for (int i = 0; i < CD_ROWS; ++i) w[i] = words{};
    if (kept) {
        sc = *reinterpret_cast<const word_mem *>(scales + (entry + my_row) * CD_BLOCKS);
#pragma unroll
        for (int i = 0; i < CD_ROWS; ++i)
            w[i] = __builtin_nontemporal_load(reinterpret_cast<const words_mem *>(codes + i * CD_APART * ROW_BYTES));
    }
    Token<T> now = read(0);

    float s[CD_ROWS][CD_COLS];
#pragma unroll
    for (int i = 0; i < CD_ROWS; ++i)
#pragma unroll
        for (int j = 0; j < CD_COLS; j += 32 / F::BITS) F::decode(w[i][j * F::BITS / 32], &s[i][j]);
    // the factors from raw numbers, which go with the first token's decay
    float factor[CD_ROWS];
    rows[wave][my_row][3] = __uint_as_float(sc);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < CD_ROWS; ++i)
        factor[i] = mx_down<F>(__float_as_uint(rows[wave][r0 + CD_APART * i][3]) >> (8 * (side / 2)) & 255);
#pragma unroll 1
    for (int32_t t = 0; t < len; ++t) {
        const float kr = to_f(now.k), qr = to_f(now.q), bt = now.beta, v0 = to_f(now.v[0]), v1 = to_f(now.v[1]);
        rows[wave][my_row] = f32x4{kr, qr, expf(now.g), 0.f};
        const float dot = OUT ? sum_half_wave(kr * qr) : 0.f;
        if (t + 1 < len) now = read(t + 1);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float kk[CD_ROWS], x[2 * CD_COLS];
#pragma unroll
        for (int i = 0; i < CD_ROWS; ++i) {
            const f32x4 row = rows[wave][r0 + CD_APART * i];
            kk[i] = row[0];
            const float decay = row[2] * factor[i];
            factor[i] = 1.f;
#pragma unroll
            for (int j = 0; j < CD_COLS; ++j) {
                s[i][j] *= decay;
                x[j] = i == 0 ? s[i][j] * row[0] : x[j] + s[i][j] * row[0];
                if (OUT) x[CD_COLS + j] = i == 0 ? s[i][j] * row[1] : x[CD_COLS + j] + s[i][j] * row[1];
            }
        }
        // over the lanes of a column.  With outputs bit 5 of the lane decides between a and
        // b, bits 4 and 3 between columns; without, the three bits between columns.
        halve32<OUT ? 16 : 8>(x);
        halve16<OUT ? 8 : 4>(x);
        halve<OUT ? 4 : 2>(x, lane & 8, [](float y) { return dpp<DPP_ROR8>(y); });
        const int buf = t & 1;
        const int bits = (lane >> 5 & 1) * 4 | (lane >> 4 & 1) * 2 | (lane >> 3 & 1);
        if (OUT)
            *reinterpret_cast<f32x4 *>(&sums[buf][wave][bits >> 2][side * CD_COLS + (bits & 3) * 4]) = f32x4{x[0], x[1], x[2], x[3]};
        else
            *reinterpret_cast<f32x2 *>(&sums[buf][wave][0][side * CD_COLS + bits * 2]) = f32x2{x[0], x[1]};
        if (OUT && lane == 0) dots[buf][wave] = dot;
        __syncthreads();   // (two buffers: a wave that is a token ahead writes to the other)
        {
            f32x2 a{}, b{};
            float qk = 0.f;
#pragma unroll
            for (int i = 0; i < CD_WAVES; ++i) {
                a += *reinterpret_cast<const f32x2 *>(&sums[buf][i][0][2 * lane]);
                if (OUT) b += *reinterpret_cast<const f32x2 *>(&sums[buf][i][1][2 * lane]), qk += dots[buf][i];
            }
            const float off0 = bt * (v0 - a[0]), off1 = bt * (v1 - a[1]);
            *reinterpret_cast<f32x2 *>(&offs[wave][2 * lane]) = f32x2{off0, off1};
            if (OUT && wave == 0) {
                typename Token<T>::two o;
                o[0] = from_f<T>(b[0] + qk * off0), o[1] = from_f<T>(b[1] + qk * off1);
                *reinterpret_cast<two_mem *>(out + ((int64_t)(t0 + t) * H + h) * CD + 2 * lane) = o;
            }
        }
        if (!write && t + 1 == len) return;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int j = 0; j < CD_COLS; ++j) {
            const float off = offs[wave][side * CD_COLS + j];
#pragma unroll
            for (int i = 0; i < CD_ROWS; ++i) s[i][j] += kk[i] * off;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    if (!write || !kept) return;
    uint32_t top[CD_ROWS], most = 0;
#pragma unroll
    for (int i = 0; i < CD_ROWS; ++i) {
        float largest = 0.f;
#pragma unroll
        for (int j = 0; j < CD_COLS; ++j) largest = mx_top(largest, s[i][j]);
        top[i] = __float_as_uint(largest) & 0x7fffffffu;   // (as bits a NaN is above all others)
        top[i] = max(top[i], dpp<DPP_XOR1>(top[i]));
        most = max(most, top[i]);
    }
    if (__any(most >= 0x7f800000u)) {   // a block without a number, hardly ever: its codes are zeros
#pragma unroll
        for (int i = 0; i < CD_ROWS; ++i)
#pragma unroll
            for (int j = 0; j < CD_COLS; ++j) s[i][j] = top[i] >= 0x7f800000u ? 0.f : s[i][j];
    }
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < CD_ROWS; ++i) {
        const int new_sc = mx_scale_of<F>(top[i]), finite = min(new_sc, 254);
        words y;
#pragma unroll
        for (int j = 0; j < WORDS; ++j) y[j] = F::encode(&s[i][j * 32 / F::BITS], finite);
        __builtin_nontemporal_store(y, reinterpret_cast<words_mem *>(codes + i * CD_APART * ROW_BYTES));
        // the row's four bytes, in all of its lanes; lane number i of a row keeps those of row i
        uint32_t bytes = (uint32_t)new_sc << (8 * (side / 2));
        bytes |= dpp<DPP_XOR2>(bytes);
        bytes |= dpp<DPP_HALF_MIRROR>(bytes);
        if (side == i) mine = bytes;
    }
    if (side < CD_ROWS) *reinterpret_cast<word_mem *>(scales + (entry + r0 + CD_APART * side) * CD_BLOCKS) = mine;
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
        // u / H = u M >> S for u < 2^24: M = (2^S + e) / H with e < H <= 2^(S - 24), so u e < 2^S
        int32_t shift = 24;
        while ((1 << (shift - 24)) < H && shift < 54) ++shift;
        const uint32_t per_head = (uint32_t)((((uint64_t)1 << shift) + H - 1) / H);
        const auto kernel = out ? kda_cached_tokens_kernel<T, decltype(f), true> : kda_cached_tokens_kernel<T, decltype(f), false>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)((int64_t)N * H)), dim3(CD_THREADS), 0, s, (const T *)q, (const T *)k,
                           (const T *)v, g, beta, cu, num_tokens, cache, scales, slots, (int32_t)write, num_slots, H,
                           per_head, shift, T_tot, (T *)out);
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

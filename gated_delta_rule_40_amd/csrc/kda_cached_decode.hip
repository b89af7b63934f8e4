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
// instructions several (token by token about 390 a wave and token for 64 values a lane:
// the decay, two products, the update, and the halving).  So a sequence of several token
// rows takes them in chunks, from one state, if there are outputs: 512 sequences of 32
// heads, fp8, two, five and eight tokens verified 88, 170 and 292 us, token by token 105, 214
// and 325; five of 64 x 16 in int8 16.6 and 18.7.  Without outputs b and the queries fall away
// and chunks gain nothing (five committed 131 us, token by token 124).
// The form goes by a sequence's own rows (cu_seqlens), not by how many of them are processed
// and not by the batch: its results have the same bits whatever stands beside it.
// One MI355X, bf16, replays of a graph: 512 sequences of 32 heads, one token committed, fp8
// 101 us (5.7 TB/s), int8 106, fp4 75; beside a sequence of five 103; 8 x 8 heads 3.8.
// Waves that each had 32 columns of all rows needed no barrier, but their reads of 32
// bytes a row bound them to 129 us; 8 columns by 8 rows a lane 119 (198 for five tokens
// verified token by token); decays kept apart from the state, as factors of its rows, gained
// 4 % for five tokens and lost 1-4 % for one; products by matrix instructions of 16 blocks
// of 4 x 4 halved the vector instructions and took 270 us for 214.
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

// A lane's part of a state, rounded and written to its codes and scales.
template <typename F> __device__ __forceinline__ void write_state(float (&s)[CD_ROWS][CD_COLS], uint8_t *codes, uint8_t *scales, int side)
{
    constexpr int WORDS = CD_COLS * F::BITS / 32, ROW_BYTES = CD * F::BITS / 8;
    typedef uint32_t words __attribute__((ext_vector_type(WORDS)));
    typedef words words_mem __attribute__((aligned(1)));
    typedef uint32_t word_mem __attribute__((aligned(1)));
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
    if (side < CD_ROWS) *reinterpret_cast<word_mem *>(scales + CD_APART * side * CD_BLOCKS) = mine;
}

// ---------------------------------------------------------------- token by token
struct TokensShared {
    f32x4 rows[CD_WAVES][CD_WROWS];                      // key, query, decay (and at first the scale bytes)
    float sums[2][CD_WAVES][2][CD], dots[2][CD_WAVES];   // of the waves: a and b; q.k
    float offs[CD_WAVES][CD];                            // a wave's own copy of beta u
};

// `len` tokens from row t0 on of head h.  OUT: with outputs (else a and the states alone).
template <typename T, typename F, bool OUT>
__device__ __forceinline__ void by_tokens(const T *q, const T *k, const T *v, const float *g, const float *beta, uint8_t *cache,
                                          uint8_t *scales, int32_t slot, int32_t write, int32_t num_slots, int32_t H, int32_t h,
                                          int32_t t0, int32_t len, T *out, TokensShared &sh)
{
    constexpr int WORDS = CD_COLS * F::BITS / 32;   // of a lane's codes in a row
    constexpr int ROW_BYTES = CD * F::BITS / 8;
    typedef uint32_t words __attribute__((ext_vector_type(WORDS)));
    typedef words words_mem __attribute__((aligned(1)));
    typedef uint32_t word_mem __attribute__((aligned(1)));
    typedef typename Token<T>::two two_mem __attribute__((aligned(sizeof(T))));
    auto &rows = sh.rows;
    auto &sums = sh.sums;
    auto &dots = sh.dots;
    auto &offs = sh.offs;

    int thread = threadIdx.x;
    asm("" : "+v"(thread));   // (places that the chunks below share with this would be held over the branch, and spilled)
    const int lane = thread & 63, wave = __builtin_amdgcn_readfirstlane(thread >> 6);
    const int side = lane % CD_LANES, r0 = lane / CD_LANES;

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
    if (write && kept) write_state<F>(s, codes, scales + (entry + r0) * CD_BLOCKS, side);
}

// without outputs
template <typename T, typename F>
__global__ __launch_bounds__(CD_THREADS, 3) void kda_cached_commit_kernel(
    const T *q, const T *k, const T *v, const float *g, const float *beta, const int32_t *cu, const int32_t *num_tokens,
    uint8_t *cache, uint8_t *scales, const int32_t *slots, int32_t write, int32_t num_slots, int32_t H,
    uint32_t per_head, int32_t shift, int32_t T_tot, T *out)
{
    const uint32_t u = blockIdx.x;
    const int32_t n = (int32_t)((uint64_t)u * per_head >> shift), h = (int32_t)u - n * H;   // u / H, u % H
    const int32_t t0 = min(max(cu[n], 0), T_tot);
    int32_t len = min(max(cu[n + 1], t0), T_tot) - t0;
    if (num_tokens) len = min(len, max(num_tokens[n], 0));
    if (len == 0) return;
    __shared__ TokensShared sh;
    by_tokens<T, F, false>(q, k, v, g, beta, cache, scales, slots[n], write, num_slots, H, h, t0, len, out, sh);
}

// ---------------------------------------------------------------- several tokens
// Up to CH tokens from one state: with c_t the decays up to token t, k_s^(t) the key of
// token s decayed up to t,
//     a_t = S^T (c_t k_t) + sum over s < t of (k_s^(t).k_t) f_s,   f_t = beta_t (v_t - a_t)
//     o_t = S^T (c_t q_t) + sum over s <= t of (k_s^(t).q_t) f_s
//     S'  = Diag(c) S + sum over s of k_s^(last) f_s^T
// so the state is multiplied by all keys and queries as it is, without a barrier between
// tokens, and moved on once (where it is only read, never).  No decay is divided by; one
// of several tokens that falls below 2^-126 keeps steps of 2^-149.
// Six tokens spill registers (five tokens 171 us for 168), eight more (178); four leave one over.
constexpr int CH = 5;

// With outputs: a sequence of one row as it is, of several by chunks.  WAVES: workgroups of a CU
// that registers are left for (four: a key's and a query's product one after the other, as both
// would spill more; 64 drafts of eight among 448 empty sequences 54 us for 77).  The results
// are the same bits.
template <typename T, typename F, int WAVES>
__global__ __launch_bounds__(CD_THREADS, WAVES) void kda_cached_outputs_kernel(
    const T *q, const T *k, const T *v, const float *g, const float *beta, const int32_t *cu, const int32_t *num_tokens,
    uint8_t *cache, uint8_t *scales, const int32_t *slots, int32_t write, int32_t num_slots, int32_t H,
    uint32_t per_head, int32_t shift, int32_t T_tot, T *out)
{
    constexpr int AT_ONCE = WAVES == 3 ? 2 : 1;     // products of the state
    constexpr int WORDS = CD_COLS * F::BITS / 32;   // of a lane's codes in a row
    constexpr int ROW_BYTES = CD * F::BITS / 8;
    typedef uint32_t words __attribute__((ext_vector_type(WORDS)));
    typedef words words_mem __attribute__((aligned(1)));
    typedef uint32_t word_mem __attribute__((aligned(1)));
    typedef typename Token<T>::two two;
    typedef two two_mem __attribute__((aligned(sizeof(T))));
    // of a wave's rows: c_t k_t and c_t q_t, then k_s^(last); c (and at first the scale bytes)
    __shared__ float rows[CD_WAVES][CH][2][CD_WROWS], ends[CD_WAVES][CD_WROWS];
    __shared__ float grams[CD_WAVES][2][CH][CH];        // a wave's part of k_s^(t).k_t and k_s^(t).q_t
    __shared__ __attribute__((aligned(16))) union {
        float sums[CH][CD_WAVES][2][CD];                // of the waves: S^T (c_t k_t), S^T (c_t q_t)
        TokensShared single;
    } sh;
    __shared__ __attribute__((aligned(16))) float offs[CH][CD];   // f_t
    auto &sums = sh.sums;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int side = lane % CD_LANES, r0 = lane / CD_LANES;
    const uint32_t u = blockIdx.x;
    const int32_t n = (int32_t)((uint64_t)u * per_head >> shift), h = (int32_t)u - n * H;   // u / H, u % H
    const int32_t t0 = min(max(cu[n], 0), T_tot);
    int32_t len = min(max(cu[n + 1], t0), T_tot) - t0;
    const bool single = len == 1;
    if (num_tokens) len = min(len, max(num_tokens[n], 0));
    const int32_t slot = slots[n];
    if (len == 0) return;
    if (single) {
        by_tokens<T, F, true>(q, k, v, g, beta, cache, scales, slot, write, num_slots, H, h, t0, 1, out, sh.single);
        return;
    }

    const int my_row = lane % CD_WROWS, query = lane / CD_WROWS;   // (keys by the lower half of a wave, queries by the upper)
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
    T kx[CH], qx[CH];
    float gx[CH], bx = 0.f;   // (beta of token t by lane t)
    two vx[CH];
    const int64_t step = (int64_t)H * CD;   // from token to token
    const auto read = [&](int32_t from) {
        const int64_t row0 = ((int64_t)(t0 + from) * H + h) * CD;
        if (lane < min(len - from, CH)) bx = beta[(int64_t)(t0 + from + lane) * H + h];
#pragma unroll
        for (int t = 0; t < CH; ++t) {
            kx[t] = qx[t] = T(0.f), gx[t] = 0.f, vx[t] = two{};
            if (t < len - from) {
                const int64_t row = row0 + t * step, at = row + wave * CD_WROWS;
                kx[t] = (k + at)[my_row], qx[t] = (q + at)[my_row], gx[t] = (g + at)[my_row];
                vx[t] = *reinterpret_cast<const two_mem *>((v + row) + 2 * lane);
            }
        }
    };
    read(0);
    float s[CD_ROWS][CD_COLS], factor[CD_ROWS];
    // the factors from raw numbers, which go with the keys and queries of the first tokens
    ends[wave][my_row] = __uint_as_float(sc);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < CD_ROWS; ++i)
        factor[i] = mx_down<F>(__float_as_uint(ends[wave][r0 + CD_APART * i]) >> (8 * (side / 2)) & 255);
#pragma unroll
    for (int i = 0; i < CD_ROWS; ++i)
#pragma unroll
        for (int j = 0; j < CD_COLS; j += 32 / F::BITS) F::decode(w[i][j * F::BITS / 32], &s[i][j]);
#pragma unroll 1
    for (int32_t from = 0;;) {
        const int32_t count = min(len - from, CH);
        const int64_t row0 = ((int64_t)(t0 + from) * H + h) * CD;
        float key[CH], c = 1.f;   // k_s^(t) of this lane's row
#pragma unroll
        for (int t = 0; t < CH; ++t) {
            if (t >= count) break;
            const float decay = expf(gx[t]), mine = query ? to_f(qx[t]) : to_f(kx[t]);
            c *= decay;
            rows[wave][t][query][my_row] = mine * c;
            float dots = 0.f;
#pragma unroll
            for (int p = 0; p <= t; ++p) {
                key[p] = p == t ? to_f(kx[t]) : key[p] * decay;
                const float dot = sum_half_wave(key[p] * mine);
                dots = my_row == p ? dot : dots;
            }
            if (my_row < CH) grams[wave][query][t][my_row] = dots;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
        for (int32_t t = 0; t < count; ++t) {
#pragma unroll 1
            for (int which = 0; which < 2; which += AT_ONCE) {   // key and query
                float x[AT_ONCE * CD_COLS];
#pragma unroll
                for (int i = 0; i < CD_ROWS; ++i)
#pragma unroll
                    for (int p = 0; p < AT_ONCE; ++p) {
                        const float r = rows[wave][t][which + p][r0 + CD_APART * i] * factor[i];
#pragma unroll
                        for (int j = 0; j < CD_COLS; ++j) {
                            float &to = x[p * CD_COLS + j];
                            to = i == 0 ? s[i][j] * r : to + s[i][j] * r;
                        }
                    }
                // over the lanes of a column, as for one token
                constexpr int LEFT = 2 * AT_ONCE;   // sums that a lane is left with
                halve32<4 * LEFT>(x);
                halve16<2 * LEFT>(x);
                halve<LEFT>(x, lane & 8, [](float y) { return dpp<DPP_ROR8>(y); });
                const int bits = (lane >> 5 & 1) * 4 | (lane >> 4 & 1) * 2 | (lane >> 3 & 1);
                typedef float left __attribute__((ext_vector_type(LEFT)));
                left y;
#pragma unroll
                for (int j = 0; j < LEFT; ++j) y[j] = x[j];
                *reinterpret_cast<left *>(AT_ONCE == 2 ? &sums[t][wave][bits >> 2][side * CD_COLS + (bits & 3) * 4]
                                                       : &sums[t][wave][which][side * CD_COLS + bits * 2]) = y;
            }
        }
        const bool moves = write || from + CH < len;
        if (moves) {   // k_s^(last) and c in the place of what the products have read
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int t = 0; t < CH; ++t)
                if (t < count) rows[wave][t][0][my_row] = key[t];
            ends[wave][my_row] = c;
        }
        __syncthreads();
        // every wave forms all f_t of two columns a lane; token t's are written by wave t % 4
        const int gram = min(lane, CH * CH - 1);
        float gk = 0.f, gq = 0.f;   // lane CH t + s: k_s^(t).k_t and .q_t
#pragma unroll
        for (int i = 0; i < CD_WAVES; ++i) gk += (&grams[i][0][0][0])[gram], gq += (&grams[i][1][0][0])[gram];
        f32x2 f[CH];
#pragma unroll
        for (int t = 0; t < CH; ++t) {
            if (t >= count) break;
            f32x2 a{};
#pragma unroll
            for (int i = 0; i < CD_WAVES; ++i) a += *reinterpret_cast<const f32x2 *>(&sums[t][i][0][2 * lane]);
            const auto lane_of = [](float x, int l) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), l)); };
#pragma unroll
            for (int p = 0; p < t; ++p) {
                const float m = lane_of(gk, CH * t + p);
                a[0] += m * f[p][0], a[1] += m * f[p][1];
            }
            const float bt = lane_of(bx, t);
            f[t] = f32x2{bt * (to_f(vx[t][0]) - a[0]), bt * (to_f(vx[t][1]) - a[1])};
            if (wave == t % CD_WAVES) {
                if (moves) *reinterpret_cast<f32x2 *>(&offs[t][2 * lane]) = f[t];
                f32x2 b{};
#pragma unroll
                for (int i = 0; i < CD_WAVES; ++i) b += *reinterpret_cast<const f32x2 *>(&sums[t][i][1][2 * lane]);
#pragma unroll
                for (int p = 0; p <= t; ++p) {
                    const float m = lane_of(gq, CH * t + p);
                    b[0] += m * f[p][0], b[1] += m * f[p][1];
                }
                two o;
                o[0] = from_f<T>(b[0]), o[1] = from_f<T>(b[1]);
                *reinterpret_cast<two_mem *>(out + row0 + t * step + 2 * lane) = o;
            }
        }
        if (!moves) return;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CD_ROWS; ++i) {
            const float decay = ends[wave][r0 + CD_APART * i] * factor[i];
            factor[i] = 1.f;
#pragma unroll
            for (int j = 0; j < CD_COLS; ++j) s[i][j] *= decay;
        }
#pragma unroll 1
        for (int32_t t = 0; t < count; ++t) {
            float kk[CD_ROWS];
#pragma unroll
            for (int i = 0; i < CD_ROWS; ++i) kk[i] = rows[wave][t][0][r0 + CD_APART * i];
#pragma unroll
            for (int j = 0; j < CD_COLS; ++j) {
                const float off = offs[t][side * CD_COLS + j];
#pragma unroll
                for (int i = 0; i < CD_ROWS; ++i) s[i][j] += kk[i] * off;
            }
        }
        from += CH;
        if (from >= len) break;
        read(from);
        __syncthreads();   // (what the next tokens write has been read)
    }
    if (write && kept) write_state<F>(s, codes, scales + (entry + r0) * CD_BLOCKS, side);
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
        typedef decltype(f) F;
        // Where no sequence need have several rows, registers for four workgroups a CU: 512 x 32, one
        // token committed, fp8 101 us (three: 103), int8 106 (116), fp4 75 (86).  The chunks spill a
        // little then: eight drafts of five, 32 heads, among 56 empty sequences 16 us (three: 12).  So
        // not where three of every CU take all sequences with a row.
        const bool three = T_tot > N || (int64_t)T_tot * H <= 3 * 256;
        const auto kernel = !out ? kda_cached_commit_kernel<T, F>
                            : three ? kda_cached_outputs_kernel<T, F, 3> : kda_cached_outputs_kernel<T, F, 4>;
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

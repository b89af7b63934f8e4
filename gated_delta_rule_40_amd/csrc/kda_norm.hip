// kda_norm.hip -- the residual's addition and root-mean-square norm of rows,
// with an output in 8 bits (e4m3 with a power-of-two scale for 32 channels),
// and its gradients.
//
//     r = x + residual,  rstd = 1 / sqrt(mean(r^2) + eps),  y = r rstd w
//     dr = rstd (w dy - r rstd^2 mean(w dy r)) + dresidual,  dw = sum_rows dy r rstd
//
// A row is held in the registers of its threads from its read to its writes,
// so every element is read once and written once, and HBM's rate is the bound.
// A row of up to 256 pieces of 16 bytes takes one wave or a part of one (no
// barrier), a longer one a workgroup.  Pieces need the alignment of an element
// only; the last one of a row may be a part of one (TAIL).
//
// Measured on one MI355X (a large copy reaches 4.9-5.4 TB/s there), bf16:
// 16,384 x 7,168 with the residual and the 8-bit output 144-147 us (5.6-5.7 TB/s
// of 7.03 bytes an element), 65,536 x 2,048 with the residual 176-179 us (6.0
// TB/s of 8 bytes), its gradients 190 us (5.7 TB/s of 8 bytes), 64 x 4,096 3.8 us.
#include "kda_colsum.hpp"
#include "kda_device.hpp"
#include "kda_layer.hpp"

#include <type_traits>

namespace kda {

constexpr int MXB = 32;              // channels that share a scale
constexpr int MAX_PARTIALS = 1024;   // partial sums of a weight's gradient

// ---------------------------------------------------------------- pieces
// VW consecutive elements, moved as one access: as read, and as fp32.  ONCE:
// past the caches, for rows too many to be found there again (65,536 x 2,048:
// 179 us, 189 through them; 16,384 x 7,168 with the 8-bit output: 147, 152); a
// few rows stay in them for the reader.
template <typename T, int VW, bool ONCE> struct Piece {
    typedef T raw __attribute__((ext_vector_type(VW)));
    typedef raw mem __attribute__((aligned(sizeof(T))));
    __device__ static __forceinline__ raw load(const T *p) {
        const mem *q = reinterpret_cast<const mem *>(p);
        return ONCE ? __builtin_nontemporal_load(q) : *q;
    }
    __device__ static __forceinline__ void store(T *p, const float (&v)[VW]) {
        raw r;
#pragma unroll
        for (int j = 0; j < VW; ++j) r[j] = from_f<T>(v[j]);
        if (ONCE) __builtin_nontemporal_store(r, reinterpret_cast<mem *>(p));
        else *reinterpret_cast<mem *>(p) = r;
    }
    // the first n elements; the others read as zeros
    __device__ static __forceinline__ raw load(const T *p, int n) {
        raw r = {};
#pragma unroll
        for (int j = 0; j < VW; ++j)
            if (j < n) r[j] = p[j];
        return r;
    }
    __device__ static __forceinline__ void store(T *p, const float (&v)[VW], int n) {
#pragma unroll
        for (int j = 0; j < VW; ++j)
            if (j < n) p[j] = from_f<T>(v[j]);
    }
    __device__ static __forceinline__ float at(const raw &r, int j) { return to_f(r[j]); }
};

// The pieces of a row of D elements, as thread i0 of its tpr has them: piece k
// is the row's number i0 + k * tpr, with `count` elements (0: beyond the row).
template <int VW, bool TAIL> struct Pieces {
    int32_t D, i0, tpr;
    __device__ __forceinline__ int32_t index(int k) const { return i0 + k * tpr; }
    __device__ __forceinline__ int32_t count(int k) const {
        const int32_t left = D - index(k) * VW;
        return TAIL ? max(min(left, VW), 0) : (left > 0 ? VW : 0);
    }
    template <typename P, typename T> __device__ __forceinline__ typename P::raw load(const T *row, int k) const {
        if (TAIL && count(k) < VW) return P::load(row + (int64_t)index(k) * VW, count(k));
        // beyond the row: the last whole piece, for nothing
        return P::load(row + min(index(k) * VW, D - VW));
    }
    template <typename P, typename T>
    __device__ __forceinline__ void store(T *row, int k, const float (&v)[VW]) const {
        const int n = count(k);
        if (n == VW) P::store(row + index(k) * VW, v);
        else if (TAIL && n > 0) P::store(row + (int64_t)index(k) * VW, v, n);
    }
    __device__ __forceinline__ void weight(const float *w, int k, float (&v)[VW]) const {
        const int n = count(k);
        const float *p = w + (int64_t)index(k) * VW;
        if (n == VW) {
            typedef f32x4 mem __attribute__((aligned(4)));
#pragma unroll
            for (int j = 0; j < VW; j += 4) {
                const f32x4 q = *reinterpret_cast<const mem *>(p + j);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j + i] = q[i];
            }
        } else {
#pragma unroll
            for (int j = 0; j < VW; ++j) v[j] = j < n ? p[j] : 0.f;
        }
    }
};

// 4 or 8 bytes at any alignment, through the caches: the product that follows
// reads them (past them 16,384 x 7,168 takes 144 us instead of 147, 100,000 x 512
// 64 instead of 63)
__device__ __forceinline__ void store_words(uint8_t *p, const uint32_t (&q)[1])
{
    typedef uint32_t mem __attribute__((aligned(1)));
    *reinterpret_cast<mem *>(p) = q[0];
}
__device__ __forceinline__ void store_words(uint8_t *p, const uint32_t (&q)[2])
{
    typedef uint32_t pair __attribute__((ext_vector_type(2)));
    typedef pair mem __attribute__((aligned(1)));
    *reinterpret_cast<mem *>(p) = pair{q[0], q[1]};
}

// Sums over a row's tpr threads (a power of two; a part of a wave, or whole
// waves).  `red` holds a value for every wave; called by the whole workgroup.
template <typename F, int M> __device__ __forceinline__ void row_sums(F (&v)[M], int tpr, F (*red)[M])
{
    for (int off = min(tpr, 64) >> 1; off > 0; off >>= 1)
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] += __shfl_xor(v[m], off);
    if (tpr <= 64) return;
    const int wave = threadIdx.x >> 6, waves = tpr >> 6, first = wave / waves * waves;
    __syncthreads();   // the row before is done with `red`
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int m = 0; m < M; ++m) red[wave][m] = v[m];
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
        F s = 0;
        for (int i = 0; i < waves; ++i) s += red[first + i][m];
        v[m] = s;
    }
}

// The e8m0 byte of a block: the smallest power of two with amax / scale <= 448
// = 0.875 * 2^9; 127 (one) for zeros, 255 (NaN) for an infinity or a NaN.
__device__ __forceinline__ int mx_scale(uint32_t amax_bits)
{
    if (amax_bits == 0) return 127;
    if (amax_bits >= 0x7f800000u) return 255;
    int e;
    const float m = frexpf(__uint_as_float(amax_bits), &e);   // amax = m 2^e, m in [1/2, 1)
    return max(e - 9 + (m > 0.875f ? 1 : 0), -127) + 127;
}

// y = r w / sqrt(mean): in fp32, which is off by up to three steps, and where
// that could matter to the 8-bit value in fp64, rounded to odd (towards zero,
// the last bit set if that is not exact), so that the next rounding is as good
// as the only one (16,384 x 7,168: none of 117 M values falls to a neighbour of
// the exact one, 60-81 with fp32 alone; exact products for every value are 7 %
// slower).
struct Rstd {
    float hi;
    double exact;
    __device__ __forceinline__ explicit Rstd(double mean) : hi(1.f / sqrtf((float)mean)), exact(hi) {
        const double off = __builtin_fma(-mean * exact, exact, 1.0);   // 1 - mean hi^2: one step to the root
        if (__builtin_fabs(off) < 1.0) exact = __builtin_fma(0.5 * exact, off, exact);   // (mean is not 0 or infinite)
    }
    __device__ __forceinline__ float times(float r, float w) const { return r * hi * w; }
    __device__ __forceinline__ float odd(float r, float w) const {
        asm("" : "+v"(r));   // (else the row stays in registers in 64 bits, from its squares on)
        const double y = (double)r * exact * w;
        const float f = (float)y;
        const double rest = y - f;
        // (`exact` is within 2^-47: a smaller rest is none)
        if (!(__builtin_fabs(rest) > 0x1p-44 * __builtin_fabs(y)) || __builtin_isinf(f)) return f;
        // (y's sign, not f's: f may be -0, from which a step back would be a NaN)
        const uint32_t bits = __float_as_uint(f), back = (rest < 0) != (y < 0);
        return __uint_as_float((bits - back) | 1u);
    }
};

// ---------------------------------------------------------------- forward
// C pieces a thread
template <typename T, int VW, int C, bool ONCE, bool TAIL, bool RES, bool MX>
__global__ void kda_rmsnorm_kernel(const T *x, const T *res, const float *w, int32_t rows, int32_t D, int32_t tpr,
                                   double per_channel, float eps, T *sum, T *out, uint8_t *mx, uint8_t *scales)
{
    typedef Piece<T, VW, ONCE> P;
    __shared__ double red[16][1];
    const Pieces<VW, TAIL> pc{D, (int32_t)(threadIdx.x & (tpr - 1)), tpr};
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = row < rows;
    const int64_t base = (live ? row : 0) * D;

    typename P::raw xr[C], rr[C];
#pragma unroll
    for (int k = 0; k < C; ++k) {
        xr[k] = pc.template load<P>(x + base, k);
        if (RES) rr[k] = pc.template load<P>(res + base, k);
    }
    float r[C][VW];
    // The squares in fp64, where each is exact: fp32 sums of eight are 1.2e-8 too
    // small on average for bf16 rows, enough for a scale in 10^8 and a value in 10^7
    // to be a neighbour of the right one (16,384 x 7,168: 146 us, 143 with them).
    double ss[1] = {0.};
#pragma unroll
    for (int k = 0; k < C; ++k) {
        double part = 0.;
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            r[k][j] = P::at(xr[k], j) + (RES ? P::at(rr[k], j) : 0.f);
            if (pc.count(k) > 0) part = __builtin_fma((double)r[k][j], (double)r[k][j], part);
        }
        ss[0] += part;
        if (RES && sum && live) pc.template store<P>(sum + base, k, r[k]);
    }
    row_sums(ss, tpr, red);
    const Rstd rstd(ss[0] * per_channel + eps);
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int32_t i = pc.index(k), n = pc.count(k);
        float g[VW], y[VW];
        if (w) pc.weight(w, k, g);
#pragma unroll
        for (int j = 0; j < VW; ++j) y[j] = rstd.times(r[k][j], w ? g[j] : 1.f);
        if (out && live) pc.template store<P>(out + base, k, y);
        if (MX) {   // a block's MXB / VW pieces lie in consecutive lanes
            auto block_top = [&]() {   // the largest of the magnitudes' bits, so that a NaN is the largest
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < VW; ++j)
                    if (j < n) top = max(top, __float_as_uint(y[j]) & 0x7fffffffu);
#pragma unroll
                for (int off = MXB / VW / 2; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
                return top;
            };
            uint32_t top = block_top();
            // within 4 steps of a tie of e4m3 (bit 19 is half a step of it) or of a
            // scale's end (448, 1.75 2^8)?  One value in 10^5 is.
            uint32_t near = (top & 0x7fffffu) - (0x600000u - 4);
#pragma unroll
            for (int j = 0; j < VW; ++j) near = min(near, (__float_as_uint(y[j]) & 0xfffffu) - (0x80000u - 4));
            // (the pieces in doubt alone: a row's bytes do not go by the rows beside it)
            if (__any(near <= 8)) {
                if (near <= 8)
#pragma unroll
                    for (int j = 0; j < VW; ++j) y[j] = rstd.odd(r[k][j], w ? g[j] : 1.f);
                top = block_top();
            }
            const int sc = mx_scale(top);
            if (n > 0 && live) {
                if (i % (MXB / VW) == 0) scales[row * ((D + MXB - 1) / MXB) + i / (MXB / VW)] = (uint8_t)sc;
                uint32_t q[VW / 4];
#pragma unroll
                for (int j = 0; j < VW; j += 4) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = ldexpf(y[j + e], 127 - sc);
                    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
                    q[j / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
                }
                uint8_t *p = mx + base + (int64_t)i * VW;
                if (n == VW) {
                    store_words(p, q);
                } else {
#pragma unroll
                    for (int j = 0; j < VW; ++j)
                        if (j < n) p[j] = (uint8_t)(q[j / 4] >> (8 * (j % 4)));
                }
            }
        }
    }
}

// ---------------------------------------------------------------- gradients
// A workgroup takes rows one after another (blockDim / tpr at a time) and keeps
// its part of the weight's gradient in registers; the parts of its rows side by
// side are added through LDS, and those of all workgroups by the next kernel,
// all in a fixed order.
template <typename T, int VW, int C, bool ONCE, bool TAIL, bool RES>
__global__ void kda_rmsnorm_bwd_kernel(const T *x, const float *w, const T *dout, const T *dres, int32_t rows,
                                       int32_t D, int32_t tpr, float eps, T *dx, float *partial)
{
    typedef Piece<T, VW, ONCE> P;
    extern __shared__ float fold[];
    __shared__ float red[16][2];
    const int i0 = threadIdx.x & (tpr - 1), slot = threadIdx.x / tpr, slots = blockDim.x / tpr;
    const Pieces<VW, TAIL> pc{D, i0, tpr};
    float dw[C][VW] = {}, g[C][VW];
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int j = 0; j < VW; ++j) g[k][j] = 1.f;
        if (w) pc.weight(w, k, g[k]);
    }
    for (int64_t row0 = (int64_t)blockIdx.x * slots; row0 < rows; row0 += (int64_t)gridDim.x * slots) {
        const int64_t row = row0 + slot;
        const bool live = row < rows;
        const int64_t base = (live ? row : row0) * D;
        typename P::raw xr[C], dr[C], rr[C];
#pragma unroll
        for (int k = 0; k < C; ++k) {
            xr[k] = pc.template load<P>(x + base, k);
            dr[k] = pc.template load<P>(dout + base, k);
            if (RES) rr[k] = pc.template load<P>(dres + base, k);
        }
        float s[2] = {0.f, 0.f};   // r^2 and w dy r
#pragma unroll
        for (int k = 0; k < C; ++k)
            if (pc.count(k) > 0)
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const float r = P::at(xr[k], j);
                    s[0] += r * r;
                    s[1] += P::at(dr[k], j) * g[k][j] * r;
                }
        row_sums(s, tpr, red);
        const float rstd = 1.f / sqrtf(s[0] / D + eps), m = s[1] / D * rstd * rstd;
#pragma unroll
        for (int k = 0; k < C; ++k) {
            float d[VW];
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                const float r = P::at(xr[k], j), dy = P::at(dr[k], j);
                d[j] = rstd * (dy * g[k][j] - m * r) + (RES ? P::at(rr[k], j) : 0.f);
                if (live) dw[k][j] += dy * (r * rstd);
            }
            if (live) pc.template store<P>(dx + base, k, d);
        }
    }
    if (!partial) return;
    // fold[slot][C * VW][tpr]: the slots' parts, added in order by the first
    if (slots > 1) {
#pragma unroll
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int j = 0; j < VW; ++j) fold[((slot * C + k) * VW + j) * tpr + i0] = dw[k][j];
        __syncthreads();
        if (slot > 0) return;
#pragma unroll
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int j = 0; j < VW; ++j)
                for (int v = 1; v < slots; ++v) dw[k][j] += fold[((v * C + k) * VW + j) * tpr + i0];
    }
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
        for (int j = 0; j < VW; ++j)
            if (j < pc.count(k)) partial[(int64_t)blockIdx.x * D + (int64_t)pc.index(k) * VW + j] = dw[k][j];
}

// dst[c] = the sum of src[i][c] over n rows
__global__ __launch_bounds__(COLSUM_THREADS) void kda_column_sums_kernel(const float *src, int32_t n, int64_t D,
                                                                         float *dst)
{
    const int64_t c = (int64_t)blockIdx.x * COLSUM_COLS + threadIdx.x % COLSUM_COLS;
    const float s = column_sum(src, n, D, c);
    if (threadIdx.x < COLSUM_COLS && c < D) dst[c] = s;
}

// ---------------------------------------------------------------- host
// Threads of a row and of a workgroup, for rows of `pieces`, at most C pieces a
// thread, and blocks of `lanes` lanes that have to lie in one row's threads.
struct RowShape {
    int tpr, threads;
};
inline RowShape row_shape(int32_t pieces, int C, int lanes)
{
    int tpr = lanes;
    while (tpr * C < pieces) tpr *= 2;
    return {tpr, tpr < 256 ? 256 : tpr};
}

// threads and workgroups of the norm at C pieces a thread
template <typename T> RowShape norm_shape(int32_t D, int C)
{
    constexpr int VW = 16 / sizeof(T);
    return row_shape((D + VW - 1) / VW, C, MXB / VW);
}
inline int64_t norm_groups(int32_t rows, const RowShape &sh)
{
    const int64_t per = sh.threads / sh.tpr;
    return (rows + per - 1) / per;
}

template <typename T, int C, bool ONCE, bool TAIL, bool RES, bool MX>
hipError_t run_rmsnorm(const void *x, const void *res, const float *w, int32_t rows, int32_t D, float eps, void *sum,
                       void *out, uint8_t *mx, uint8_t *scales, hipStream_t s)
{
    constexpr int VW = 16 / sizeof(T);
    const RowShape sh = norm_shape<T>(D, C);
    hipLaunchKernelGGL((kda_rmsnorm_kernel<T, VW, C, ONCE, TAIL, RES, MX>), dim3((unsigned)norm_groups(rows, sh)),
                       dim3(sh.threads), 0, s, (const T *)x, (const T *)res, w, rows, D, sh.tpr, 1.0 / D, eps, (T *)sum, (T *)out, mx,
                       scales);
    return hipGetLastError();
}

template <typename T, int C, bool ONCE, bool TAIL>
hipError_t rmsnorm_as(const void *x, const void *res, const float *w, int32_t rows, int32_t D, float eps, void *sum,
                      void *out, uint8_t *mx, uint8_t *scales, hipStream_t s)
{
    if (res)
        return mx ? run_rmsnorm<T, C, ONCE, TAIL, true, true>(x, res, w, rows, D, eps, sum, out, mx, scales, s)
                  : run_rmsnorm<T, C, ONCE, TAIL, true, false>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
    return mx ? run_rmsnorm<T, C, ONCE, TAIL, false, true>(x, res, w, rows, D, eps, sum, out, mx, scales, s)
              : run_rmsnorm<T, C, ONCE, TAIL, false, false>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
}

// calls f with the number of pieces a thread, whether rows go past the caches,
// and whether they end in a part of a piece, as compile-time values.  Few rows:
// one piece a thread, so that a row's latency is short (64 x 4,096: 3.3 us, 4.5
// with four; 512 x 7,168: 7.1, 6.9); and for short rows, so that a row has
// threads enough (200,000 x 128: 35 us, 56 with four; 100,000 x 512: 68, 71).
template <typename T, int MOST, typename F> auto with_shape(int32_t rows, int32_t D, F f)
{
    constexpr int VW = 16 / sizeof(T);
    const int32_t pieces = (D + VW - 1) / VW;
    auto tail = [&](auto c, auto once) {
        return D % VW ? f(c, once, std::true_type()) : f(c, once, std::false_type());
    };
    const std::integral_constant<int, 1> one;
    if (rows <= 512 && pieces <= 1024) return tail(one, std::false_type());
    if (pieces <= 64) return tail(one, std::true_type());
    return tail(std::integral_constant<int, MOST>(), std::true_type());
}

template <typename T> bool rmsnorm_fits(int32_t rows, int32_t D)
{
    return with_shape<T, 4>(rows, D, [&](auto c, auto, auto) {
        const RowShape sh = norm_shape<T>(D, c());
        return kda_grid_ok(norm_groups(rows, sh), sh.threads);
    });
}

template <typename T>
hipError_t rmsnorm(const void *x, const void *res, const float *w, int32_t rows, int32_t D, float eps, void *sum,
                   void *out, uint8_t *mx, uint8_t *scales, hipStream_t s)
{
    return with_shape<T, 4>(rows, D, [&](auto c, auto once, auto tail) {
        return rmsnorm_as<T, c(), once(), tail()>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
    });
}

inline int32_t partials(int32_t rows) { return rows < MAX_PARTIALS ? rows : MAX_PARTIALS; }

template <typename T, int C, bool ONCE, bool TAIL>
hipError_t rmsnorm_backward_as(const void *x, const float *w, const void *dout, const void *dres, int32_t rows,
                               int32_t D, float eps, void *dx, float *dw, void *ws, hipStream_t s)
{
    constexpr int VW = 16 / sizeof(T);
    const RowShape sh = row_shape((D + VW - 1) / VW, C, 1);
    const int64_t per = sh.threads / sh.tpr, groups = (rows + per - 1) / per;
    const unsigned blocks = (unsigned)(groups < MAX_PARTIALS ? groups : MAX_PARTIALS);
    const size_t lds = per > 1 ? sizeof(float) * sh.threads * C * VW : 0;
    if (blocks > 0) {
        if (dres)
            hipLaunchKernelGGL((kda_rmsnorm_bwd_kernel<T, VW, C, ONCE, TAIL, true>), dim3(blocks), dim3(sh.threads),
                               lds, s, (const T *)x, w, (const T *)dout, (const T *)dres, rows, D, sh.tpr, eps,
                               (T *)dx, dw ? (float *)ws : nullptr);
        else
            hipLaunchKernelGGL((kda_rmsnorm_bwd_kernel<T, VW, C, ONCE, TAIL, false>), dim3(blocks), dim3(sh.threads),
                               lds, s, (const T *)x, w, (const T *)dout, (const T *)dres, rows, D, sh.tpr, eps,
                               (T *)dx, dw ? (float *)ws : nullptr);
    }
    if (dw)
        hipLaunchKernelGGL(kda_column_sums_kernel, dim3((unsigned)((D + COLSUM_COLS - 1) / COLSUM_COLS)),
                           dim3(COLSUM_THREADS), 0, s, (const float *)ws, (int32_t)blocks, (int64_t)D, dw);
    return hipGetLastError();
}

template <typename T>
hipError_t rmsnorm_backward(const void *x, const float *w, const void *dout, const void *dres, int32_t rows, int32_t D,
                            float eps, void *dx, float *dw, void *ws, hipStream_t s)
{
    // two pieces of eight or four of four: more would not fit the registers
    return with_shape<T, (int)sizeof(T)>(rows, D, [&](auto c, auto once, auto tail) {
        return rmsnorm_backward_as<T, c(), once(), tail()>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s);
    });
}

}  // namespace kda

using namespace kda;

bool kda_rmsnorm_fits(bool bf16, int32_t rows, int32_t D)
{
    return bf16 ? rmsnorm_fits<bf16_t>(rows, D) : rmsnorm_fits<float>(rows, D);
}

hipError_t kda_launch_rmsnorm(bool bf16, const void *x, const void *residual, const float *w, int32_t rows, int32_t D,
                              float eps, void *sum, void *out, uint8_t *mx, uint8_t *scales, hipStream_t s)
{
    return bf16 ? rmsnorm<bf16_t>(x, residual, w, rows, D, eps, sum, out, mx, scales, s)
                : rmsnorm<float>(x, residual, w, rows, D, eps, sum, out, mx, scales, s);
}

size_t kda_rmsnorm_bwd_ws_bytes(int32_t rows, int32_t D) { return (size_t)partials(rows) * D * sizeof(float); }

hipError_t kda_launch_rmsnorm_backward(bool bf16, const void *x, const float *w, const void *dout, const void *dres,
                                       int32_t rows, int32_t D, float eps, void *dx, float *dw, void *ws,
                                       hipStream_t s)
{
    return bf16 ? rmsnorm_backward<bf16_t>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s)
                : rmsnorm_backward<float>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s);
}

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
// barrier), a longer one a workgroup.  Where a row's channels or pointers are
// no multiples of 16 bytes, single elements stand for the pieces.
#include "kda_colsum.hpp"
#include "kda_device.hpp"
#include "kda_layer.hpp"

namespace kda {

constexpr int MXB = 32;              // channels that share a scale
constexpr int MAX_PARTIALS = 1024;   // partial sums of a weight's gradient

// ---------------------------------------------------------------- pieces
// VW consecutive elements, moved as one access: as read, and as fp32.  ONCE:
// past the caches, for rows too many to be found there again (16,384 x 7,168
// with the 8-bit output 152 -> 135 us); a few rows stay in them for the reader.
template <typename T, int VW, bool ONCE> struct Piece {
    typedef T raw __attribute__((ext_vector_type(VW)));
    __device__ static __forceinline__ raw load(const T *p) {
        const raw *q = reinterpret_cast<const raw *>(p);
        return ONCE ? __builtin_nontemporal_load(q) : *q;
    }
    __device__ static __forceinline__ void store(T *p, const float (&v)[VW]) {
        raw r;
#pragma unroll
        for (int j = 0; j < VW; ++j) r[j] = from_f<T>(v[j]);
        if (ONCE) __builtin_nontemporal_store(r, reinterpret_cast<raw *>(p));
        else *reinterpret_cast<raw *>(p) = r;
    }
    __device__ static __forceinline__ float at(const raw &r, int j) { return to_f(r[j]); }
};
template <typename T, bool ONCE> struct Piece<T, 1, ONCE> {
    typedef T raw;
    __device__ static __forceinline__ raw load(const T *p) { return *p; }
    __device__ static __forceinline__ void store(T *p, const float (&v)[1]) { *p = from_f<T>(v[0]); }
    __device__ static __forceinline__ float at(const raw &r, int) { return to_f(r); }
};
template <int VW> __device__ __forceinline__ void load_weight(const float *w, int64_t c, float (&v)[VW])
{
    if (VW % 4 == 0) {
#pragma unroll
        for (int j = 0; j < VW; j += 4) {
            const f32x4 q = *reinterpret_cast<const f32x4 *>(w + c + j);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j + i] = q[i];
        }
    } else {
#pragma unroll
        for (int j = 0; j < VW; ++j) v[j] = w[c + j];
    }
}

// Sums over a row's tpr threads (a power of two; a part of a wave, or whole
// waves).  `red` holds a value for every wave; called by the whole workgroup.
template <int M> __device__ __forceinline__ void row_sums(float (&v)[M], int tpr, float (*red)[M])
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
        float s = 0.f;
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

// ---------------------------------------------------------------- forward
// Pieces of a row: thread i of its tpr has pieces i, i + tpr, ... (C of them).
template <typename T, int VW, int C, bool ONCE, bool RES, bool MX>
__global__ void kda_rmsnorm_kernel(const T *x, const T *res, const float *w, int32_t rows, int32_t D, int32_t tpr,
                                   float eps, T *sum, T *out, uint8_t *mx, uint8_t *scales)
{
    typedef Piece<T, VW, ONCE> P;
    __shared__ float red[16][1];
    const int i0 = threadIdx.x & (tpr - 1);
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = row < rows;
    const int64_t base = (live ? row : 0) * D;
    const int32_t pieces = D / VW;

    typename P::raw xr[C], rr[C];
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int32_t i = min(i0 + k * tpr, pieces - 1);
        xr[k] = P::load(x + base + (int64_t)i * VW);
        if (RES) rr[k] = P::load(res + base + (int64_t)i * VW);
    }
    float r[C][VW], ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const bool have = i0 + k * tpr < pieces;
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            r[k][j] = P::at(xr[k], j) + (RES ? P::at(rr[k], j) : 0.f);
            if (have) ss[0] += r[k][j] * r[k][j];
        }
        if (RES && sum && have && live) P::store(sum + base + (int64_t)(i0 + k * tpr) * VW, r[k]);
    }
    row_sums<1>(ss, tpr, red);
    const float rstd = 1.f / sqrtf(ss[0] / D + eps);
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int32_t i = i0 + k * tpr;
        const bool have = i < pieces;
        float g[VW];
        if (w) load_weight<VW>(w, (int64_t)min(i, pieces - 1) * VW, g);
#pragma unroll
        for (int j = 0; j < VW; ++j) r[k][j] = r[k][j] * rstd * (w ? g[j] : 1.f);
        if (out && have && live) P::store(out + base + (int64_t)i * VW, r[k]);
        if (MX) {   // a block's MXB / VW pieces lie in consecutive lanes
            uint32_t top = 0;   // of the magnitudes' bits, so that a NaN is the largest
#pragma unroll
            for (int j = 0; j < VW; ++j) top = max(top, __float_as_uint(r[k][j]) & 0x7fffffffu);
            if (!have) top = 0;
#pragma unroll
            for (int off = MXB / VW / 2; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
            const int sc = mx_scale(top);
            if (have && live) {
                if (i % (MXB / VW) == 0) scales[row * ((D + MXB - 1) / MXB) + i / (MXB / VW)] = (uint8_t)sc;
                float q[VW];
#pragma unroll
                for (int j = 0; j < VW; ++j) q[j] = ldexpf(r[k][j], 127 - sc);
                uint8_t *p = mx + base + (int64_t)i * VW;
                if (VW == 1) {
                    *p = (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[0], 0, false) & 0xff);
                } else {
                    uint32_t word[VW >= 4 ? VW / 4 : 1];
#pragma unroll
                    for (int j = 0; j + 3 < VW; j += 4) {
                        int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[j], q[j + 1], 0, false);
                        word[j / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[j + 2], q[j + 3], v, true);
                    }
                    if (VW == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(word[0], word[VW >= 8 ? 1 : 0]);
                    else *reinterpret_cast<uint32_t *>(p) = word[0];
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
template <typename T, int VW, int C, bool ONCE, bool RES>
__global__ void kda_rmsnorm_bwd_kernel(const T *x, const float *w, const T *dout, const T *dres, int32_t rows,
                                       int32_t D, int32_t tpr, float eps, T *dx, float *partial)
{
    typedef Piece<T, VW, ONCE> P;
    extern __shared__ float fold[];
    __shared__ float red[16][2];
    const int i0 = threadIdx.x & (tpr - 1), slot = threadIdx.x / tpr, slots = blockDim.x / tpr;
    const int32_t pieces = D / VW;
    float dw[C][VW] = {}, g[C][VW];
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int j = 0; j < VW; ++j) g[k][j] = 1.f;
        if (w) load_weight<VW>(w, (int64_t)min(i0 + k * tpr, pieces - 1) * VW, g[k]);
    }
    for (int64_t row0 = (int64_t)blockIdx.x * slots; row0 < rows; row0 += (int64_t)gridDim.x * slots) {
        const int64_t row = row0 + slot;
        const bool live = row < rows;
        const int64_t base = (live ? row : row0) * D;
        typename P::raw xr[C], dr[C], rr[C];
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int64_t at = base + (int64_t)min(i0 + k * tpr, pieces - 1) * VW;
            xr[k] = P::load(x + at);
            dr[k] = P::load(dout + at);
            if (RES) rr[k] = P::load(dres + at);
        }
        float s[2] = {0.f, 0.f};   // r^2 and w dy r
#pragma unroll
        for (int k = 0; k < C; ++k)
            if (i0 + k * tpr < pieces)
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    const float r = P::at(xr[k], j);
                    s[0] += r * r;
                    s[1] += P::at(dr[k], j) * g[k][j] * r;
                }
        row_sums<2>(s, tpr, red);
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
            if (live && i0 + k * tpr < pieces) P::store(dx + base + (int64_t)(i0 + k * tpr) * VW, d);
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
        if (i0 + k * tpr < pieces)
#pragma unroll
            for (int j = 0; j < VW; ++j) partial[(int64_t)blockIdx.x * D + (int64_t)(i0 + k * tpr) * VW + j] = dw[k][j];
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
inline bool on(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

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

template <typename T, int VW, int C, bool ONCE, bool RES, bool MX>
hipError_t run_rmsnorm(const void *x, const void *res, const float *w, int32_t rows, int32_t D, float eps, void *sum,
                       void *out, uint8_t *mx, uint8_t *scales, hipStream_t s)
{
    const RowShape sh = row_shape(D / VW, C, MXB / VW);
    const int64_t per = sh.threads / sh.tpr;
    hipLaunchKernelGGL((kda_rmsnorm_kernel<T, VW, C, ONCE, RES, MX>), dim3((unsigned)((rows + per - 1) / per)),
                       dim3(sh.threads), 0, s, (const T *)x, (const T *)res, w, rows, D, sh.tpr, eps, (T *)sum,
                       (T *)out, mx, scales);
    return hipGetLastError();
}

template <typename T, int VW, int C, bool ONCE>
hipError_t rmsnorm_as(const void *x, const void *res, const float *w, int32_t rows, int32_t D, float eps, void *sum,
                      void *out, uint8_t *mx, uint8_t *scales, hipStream_t s)
{
    if (res)
        return mx ? run_rmsnorm<T, VW, C, ONCE, true, true>(x, res, w, rows, D, eps, sum, out, mx, scales, s)
                  : run_rmsnorm<T, VW, C, ONCE, true, false>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
    return mx ? run_rmsnorm<T, VW, C, ONCE, false, true>(x, res, w, rows, D, eps, sum, out, mx, scales, s)
              : run_rmsnorm<T, VW, C, ONCE, false, false>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
}

template <typename T>
hipError_t rmsnorm(const void *x, const void *res, const float *w, int32_t rows, int32_t D, float eps, void *sum,
                   void *out, uint8_t *mx, uint8_t *scales, hipStream_t s)
{
    constexpr int VW = 16 / sizeof(T);
    if (D % VW == 0 && on(x, 16) && on(res, 16) && on(w, 16) && on(sum, 16) && on(out, 16) && on(mx, VW)) {
        const int32_t pieces = D / VW;
        // few rows: one piece a thread, so that a row's latency is short
        if (rows <= 512 && pieces <= 1024)
            return rmsnorm_as<T, VW, 1, false>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
        if (pieces <= 64) return rmsnorm_as<T, VW, 1, true>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
        return rmsnorm_as<T, VW, 4, true>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
    }
    if (D <= 4096) return rmsnorm_as<T, 1, 4, false>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
    return rmsnorm_as<T, 1, 16, false>(x, res, w, rows, D, eps, sum, out, mx, scales, s);
}

inline int32_t partials(int32_t rows) { return rows < MAX_PARTIALS ? rows : MAX_PARTIALS; }

template <typename T, int VW, int C, bool ONCE>
hipError_t rmsnorm_backward_as(const void *x, const float *w, const void *dout, const void *dres, int32_t rows,
                               int32_t D, float eps, void *dx, float *dw, void *ws, hipStream_t s)
{
    const RowShape sh = row_shape(D / VW, C, 1);
    const int64_t per = sh.threads / sh.tpr, groups = (rows + per - 1) / per;
    const unsigned blocks = (unsigned)(groups < MAX_PARTIALS ? groups : MAX_PARTIALS);
    const size_t lds = per > 1 ? sizeof(float) * sh.threads * C * VW : 0;
    if (blocks > 0) {
        if (dres)
            hipLaunchKernelGGL((kda_rmsnorm_bwd_kernel<T, VW, C, ONCE, true>), dim3(blocks), dim3(sh.threads), lds, s,
                               (const T *)x, w, (const T *)dout, (const T *)dres, rows, D, sh.tpr, eps, (T *)dx,
                               dw ? (float *)ws : nullptr);
        else
            hipLaunchKernelGGL((kda_rmsnorm_bwd_kernel<T, VW, C, ONCE, false>), dim3(blocks), dim3(sh.threads), lds, s,
                               (const T *)x, w, (const T *)dout, (const T *)dres, rows, D, sh.tpr, eps, (T *)dx,
                               dw ? (float *)ws : nullptr);
    }
    if (dw)
        hipLaunchKernelGGL(kda_column_sums_kernel, dim3((unsigned)((D + COLSUM_COLS - 1) / COLSUM_COLS)),
                           dim3(COLSUM_THREADS), 0, s,
                           (const float *)ws, (int32_t)blocks, (int64_t)D, dw);
    return hipGetLastError();
}

template <typename T>
hipError_t rmsnorm_backward(const void *x, const float *w, const void *dout, const void *dres, int32_t rows, int32_t D,
                            float eps, void *dx, float *dw, void *ws, hipStream_t s)
{
    constexpr int VW = 16 / sizeof(T);
    if (D % VW == 0 && on(x, 16) && on(dout, 16) && on(dres, 16) && on(w, 16) && on(dx, 16)) {
        const int32_t pieces = D / VW;
        if (rows <= 512 && pieces <= 1024)
            return rmsnorm_backward_as<T, VW, 1, false>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s);
        if (pieces <= 64) return rmsnorm_backward_as<T, VW, 1, true>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s);
        // two pieces of eight or four of four: more would not fit the registers
        return rmsnorm_backward_as<T, VW, 16 / VW, true>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s);
    }
    if (D <= 4096) return rmsnorm_backward_as<T, 1, 4, false>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s);
    return rmsnorm_backward_as<T, 1, 16, false>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s);
}

}  // namespace kda

using namespace kda;

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

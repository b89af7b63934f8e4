// kda_norm.hip -- the residual's addition and root-mean-square norm of rows,
// with an output in 8 bits (e4m3 with a power-of-two scale for 32 channels),
// and its gradients.
//
// One workgroup per row.
#include "kda_device.hpp"
#include "kda_layer.hpp"

namespace kda {

constexpr int NT = 256;
constexpr int MXB = 32;   // channels that share a scale

__device__ __forceinline__ float block_sum(float v, float *red)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < NT / 64; ++i) s += red[i];
    return s;
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

template <typename T>
__global__ void kda_rmsnorm_kernel(const T *x, const T *res, const float *w, int32_t D, float eps, T *sum, T *out,
                                   uint8_t *mx, uint8_t *scales)
{
    extern __shared__ float row[];
    __shared__ float red[NT / 64];
    const int64_t base = (int64_t)blockIdx.x * D;
    float ss = 0.f;
    for (int c = threadIdx.x; c < D; c += NT) {
        float r = to_f(x[base + c]);
        if (res) r += to_f(res[base + c]);
        if (sum) sum[base + c] = from_f<T>(r);
        row[c] = r;
        ss += r * r;
    }
    const float rstd = 1.f / sqrtf(block_sum(ss, red) / D + eps);
    for (int c = threadIdx.x; c < D; c += NT) {
        const float y = row[c] * rstd * (w ? w[c] : 1.f);
        row[c] = y;
        if (out) out[base + c] = from_f<T>(y);
    }
    if (!mx) return;
    __syncthreads();
    const int nb = (D + MXB - 1) / MXB;
    for (int b = threadIdx.x; b < nb; b += NT) {
        uint32_t top = 0;   // of the magnitudes' bits, so that a NaN is the largest
        for (int c = b * MXB; c < min(D, (b + 1) * MXB); ++c) top = max(top, __float_as_uint(row[c]) & 0x7fffffffu);
        const int sc = mx_scale(top);
        scales[(int64_t)blockIdx.x * nb + b] = (uint8_t)sc;
        for (int c = b * MXB; c < min(D, (b + 1) * MXB); ++c) {
            const float q = sc == 255 ? row[c] : ldexpf(row[c], 127 - sc);
            mx[base + c] = (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false) & 0xff);
        }
    }
}

template <typename T>
__global__ void kda_rmsnorm_bwd_kernel(const T *x, const float *w, const T *dout, const T *dres, int32_t D, float eps,
                                       T *dx)
{
    __shared__ float red[NT / 64];
    const int64_t base = (int64_t)blockIdx.x * D;
    float ss = 0.f, dot = 0.f;
    for (int c = threadIdx.x; c < D; c += NT) {
        const float r = to_f(x[base + c]);
        ss += r * r;
        dot += to_f(dout[base + c]) * (w ? w[c] : 1.f) * r;
    }
    const float rstd = 1.f / sqrtf(block_sum(ss, red) / D + eps);
    const float k = block_sum(dot, red) / D * rstd * rstd;
    for (int c = threadIdx.x; c < D; c += NT) {
        float d = rstd * (to_f(dout[base + c]) * (w ? w[c] : 1.f) - k * to_f(x[base + c]));
        if (dres) d += to_f(dres[base + c]);
        dx[base + c] = from_f<T>(d);
    }
}

// the rows' 1 / rms, before dx may take x's place
template <typename T>
__global__ void kda_rmsnorm_rstd_kernel(const T *x, int32_t D, float eps, float *rstd)
{
    __shared__ float red[NT / 64];
    const int64_t base = (int64_t)blockIdx.x * D;
    float ss = 0.f;
    for (int c = threadIdx.x; c < D; c += NT) {
        const float r = to_f(x[base + c]);
        ss += r * r;
    }
    const float s = block_sum(ss, red);
    if (threadIdx.x == 0) rstd[blockIdx.x] = 1.f / sqrtf(s / D + eps);
}

template <typename T>
__global__ void kda_rmsnorm_dw_kernel(const T *x, const T *dout, const float *rstd, int32_t rows, int32_t D, float *dw)
{
    const int32_t c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= D) return;
    float s = 0.f;
    for (int32_t i = 0; i < rows; ++i) s += to_f(dout[(int64_t)i * D + c]) * to_f(x[(int64_t)i * D + c]) * rstd[i];
    dw[c] = s;
}

template <typename T>
hipError_t launch_rmsnorm(const void *x, const void *res, const float *w, int32_t rows, int32_t D, float eps,
                          void *sum, void *out, uint8_t *mx, uint8_t *scales, hipStream_t s)
{
    static std::atomic<uint64_t> done{0};
    if (hipError_t e = ensure_lds_limit((const void *)kda_rmsnorm_kernel<T>, kMaxNormChannels * 4, done)) return e;
    hipLaunchKernelGGL(kda_rmsnorm_kernel<T>, dim3(rows), dim3(NT), D * sizeof(float), s, (const T *)x,
                       (const T *)res, w, D, eps, (T *)sum, (T *)out, mx, scales);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_rmsnorm_backward(const void *x, const float *w, const void *dout, const void *dres, int32_t rows,
                                   int32_t D, float eps, void *dx, float *dw, void *ws, hipStream_t s)
{
    if (dw) {
        if (rows > 0)
            hipLaunchKernelGGL(kda_rmsnorm_rstd_kernel<T>, dim3(rows), dim3(NT), 0, s, (const T *)x, D, eps,
                               (float *)ws);
        hipLaunchKernelGGL(kda_rmsnorm_dw_kernel<T>, dim3((D + 63) / 64), dim3(64), 0, s, (const T *)x,
                           (const T *)dout, (const float *)ws, rows, D, dw);
    }
    if (rows > 0)
        hipLaunchKernelGGL(kda_rmsnorm_bwd_kernel<T>, dim3(rows), dim3(NT), 0, s, (const T *)x, w, (const T *)dout,
                           (const T *)dres, D, eps, (T *)dx);
    return hipGetLastError();
}

}  // namespace kda

using namespace kda;

hipError_t kda_launch_rmsnorm(bool bf16, const void *x, const void *residual, const float *w, int32_t rows, int32_t D,
                              float eps, void *sum, void *out, uint8_t *mx, uint8_t *scales, hipStream_t s)
{
    return bf16 ? launch_rmsnorm<bf16_t>(x, residual, w, rows, D, eps, sum, out, mx, scales, s)
                : launch_rmsnorm<float>(x, residual, w, rows, D, eps, sum, out, mx, scales, s);
}

size_t kda_rmsnorm_bwd_ws_bytes(int32_t rows, int32_t) { return (size_t)rows * sizeof(float); }

hipError_t kda_launch_rmsnorm_backward(bool bf16, const void *x, const float *w, const void *dout, const void *dres,
                                       int32_t rows, int32_t D, float eps, void *dx, float *dw, void *ws,
                                       hipStream_t s)
{
    return bf16 ? launch_rmsnorm_backward<bf16_t>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s)
                : launch_rmsnorm_backward<float>(x, w, dout, dres, rows, D, eps, dx, dw, ws, s);
}

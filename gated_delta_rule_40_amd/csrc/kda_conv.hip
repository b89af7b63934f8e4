// kda_conv.hip -- short causal convolution over the tokens of packed
// sequences, per channel, with an optional SiLU; its decode step and gradients.
//
// One thread per (token, channel).
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_seq.hpp"

namespace kda {

constexpr int MAXW = 4;

struct ConvArgs {
    const float *w, *bias;
    int32_t D, width;
    bool silu;
};

__device__ __forceinline__ float silu_f(float p) { return p / (1.f + expf(-p)); }
__device__ __forceinline__ float dsilu_f(float p)
{
    const float sig = 1.f / (1.f + expf(-p));
    return sig * (1.f + p * (1.f - sig));
}

// input at place p (from -(width - 1)) of sequence n, which starts at token t0
template <typename T>
__device__ __forceinline__ float conv_input(const T *x, const T *init, const ConvArgs &a, int32_t n, int32_t t0,
                                            int32_t p, int32_t c)
{
    if (p >= 0) return to_f(x[(int64_t)(t0 + p) * a.D + c]);
    return init ? to_f(init[((int64_t)n * (a.width - 1) + a.width - 1 + p) * a.D + c]) : 0.f;
}

template <typename T>
__device__ __forceinline__ float conv_pre(const T *x, const T *init, const ConvArgs &a, int32_t n, int32_t t0,
                                          int32_t p, int32_t c)
{
    float s = a.bias ? a.bias[c] : 0.f;
    for (int j = 0; j < a.width; ++j)
        s += a.w[(int64_t)c * a.width + j] * conv_input(x, init, a, n, t0, p - (a.width - 1) + j, c);
    return s;
}

template <typename T>
__global__ void kda_conv_kernel(const T *x, const T *init, ConvArgs a, Seqs sq, T *out)
{
    const int64_t total = (int64_t)sq.T * a.D;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int32_t t = (int32_t)(i / a.D), c = (int32_t)(i % a.D), n = sq.owner(t);
        if (n < 0) continue;
        const int32_t t0 = sq.at(n);
        const float p = conv_pre(x, init, a, n, t0, t - t0, c);
        out[i] = from_f<T>(a.silu ? silu_f(p) : p);
    }
}

// final_state, after the outputs: it may take initial_state's place
template <typename T>
__global__ void kda_conv_final_kernel(const T *x, const T *init, ConvArgs a, Seqs sq, T *fin)
{
    const int64_t total = (int64_t)sq.N * a.D;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int32_t n = (int32_t)(i / a.D), c = (int32_t)(i % a.D), t0 = sq.at(n);
        const int32_t len = max(sq.at(n + 1) - t0, 0);
        float v[MAXW - 1];
        for (int j = 0; j < a.width - 1; ++j) v[j] = conv_input(x, init, a, n, t0, len - (a.width - 1) + j, c);
        for (int j = 0; j < a.width - 1; ++j) fin[((int64_t)n * (a.width - 1) + j) * a.D + c] = from_f<T>(v[j]);
    }
}

template <typename T>
__global__ void kda_conv_step_kernel(const T *x, T *state, ConvArgs a, int32_t N, T *out)
{
    const int64_t total = (int64_t)N * a.D;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int32_t n = (int32_t)(i / a.D), c = (int32_t)(i % a.D);
        T *st = state + (int64_t)n * (a.width - 1) * a.D + c;
        T v[MAXW];
        for (int j = 0; j < a.width - 1; ++j) v[j] = st[(int64_t)j * a.D];
        v[a.width - 1] = x[i];
        float p = a.bias ? a.bias[c] : 0.f;
        for (int j = 0; j < a.width; ++j) p += a.w[(int64_t)c * a.width + j] * to_f(v[j]);
        for (int j = 0; j < a.width - 1; ++j) st[(int64_t)j * a.D] = v[j + 1];
        out[i] = from_f<T>(a.silu ? silu_f(p) : p);
    }
}

// gradient of pre at place p of sequence n
template <typename T>
__device__ __forceinline__ float conv_dpre(const T *x, const T *init, const ConvArgs &a, const T *dout, int32_t n,
                                           int32_t t0, int32_t p, int32_t c)
{
    const float d = to_f(dout[(int64_t)(t0 + p) * a.D + c]);
    return a.silu ? d * dsilu_f(conv_pre(x, init, a, n, t0, p, c)) : d;
}

// gradient of the input at place p (from -(width - 1)) of sequence n of length len
template <typename T>
__device__ __forceinline__ float conv_dinput(const T *x, const T *init, const ConvArgs &a, const T *dout,
                                             const T *dfinal, int32_t n, int32_t t0, int32_t len, int32_t p, int32_t c)
{
    float s = 0.f;
    for (int k = 0; k < a.width; ++k) {
        const int32_t q = p + k;
        if (q >= 0 && q < len)
            s += a.w[(int64_t)c * a.width + a.width - 1 - k] * conv_dpre(x, init, a, dout, n, t0, q, c);
    }
    const int32_t j = p - (len - (a.width - 1));   // its place in the final state
    if (dfinal && j >= 0) s += to_f(dfinal[((int64_t)n * (a.width - 1) + j) * a.D + c]);
    return s;
}

template <typename T>
__global__ void kda_conv_bwd_dx_kernel(const T *x, const T *init, ConvArgs a, Seqs sq, const T *dout, const T *dfinal,
                                       T *dx)
{
    const int64_t total = (int64_t)sq.T * a.D;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int32_t t = (int32_t)(i / a.D), c = (int32_t)(i % a.D), n = sq.owner(t);
        if (n < 0) continue;
        const int32_t t0 = sq.at(n), len = max(sq.at(n + 1) - t0, 0);
        dx[i] = from_f<T>(conv_dinput(x, init, a, dout, dfinal, n, t0, len, t - t0, c));
    }
}

template <typename T>
__global__ void kda_conv_bwd_dinit_kernel(const T *x, const T *init, ConvArgs a, Seqs sq, const T *dout,
                                          const T *dfinal, T *dinit)
{
    const int64_t total = (int64_t)sq.N * (a.width - 1) * a.D;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int32_t c = (int32_t)(i % a.D), j = (int32_t)(i / a.D % (a.width - 1));
        const int32_t n = (int32_t)(i / a.D / (a.width - 1)), t0 = sq.at(n), len = max(sq.at(n + 1) - t0, 0);
        dinit[i] = from_f<T>(conv_dinput(x, init, a, dout, dfinal, n, t0, len, j - (a.width - 1), c));
    }
}

template <typename T>
__global__ void kda_conv_bwd_dw_kernel(const T *x, const T *init, ConvArgs a, Seqs sq, const T *dout, float *dw,
                                       float *dbias)
{
    const int32_t c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= a.D) return;
    float s[MAXW] = {}, b = 0.f;
    for (int32_t n = 0; n < sq.N; ++n) {
        const int32_t t0 = sq.at(n), len = max(sq.at(n + 1) - t0, 0);
        for (int32_t p = 0; p < len; ++p) {
            const float d = conv_dpre(x, init, a, dout, n, t0, p, c);
            b += d;
            for (int j = 0; j < a.width; ++j) s[j] += d * conv_input(x, init, a, n, t0, p - (a.width - 1) + j, c);
        }
    }
    for (int j = 0; j < a.width; ++j) dw[(int64_t)c * a.width + j] = s[j];
    if (dbias) dbias[c] = b;
}

inline unsigned conv_blocks(int64_t n, int per)
{
    const int64_t b = (n + per - 1) / per;
    return (unsigned)(b < (1 << 20) ? b : (1 << 20));
}

template <typename T>
hipError_t launch_conv(const void *x, const ConvArgs &a, const void *init, const Seqs &sq, void *out, void *fin,
                       hipStream_t s)
{
    if (sq.T > 0)
        hipLaunchKernelGGL(kda_conv_kernel<T>, dim3(conv_blocks((int64_t)sq.T * a.D, 256)), dim3(256), 0, s,
                           (const T *)x, (const T *)init, a, sq, (T *)out);
    if (fin)
        hipLaunchKernelGGL(kda_conv_final_kernel<T>, dim3(conv_blocks((int64_t)sq.N * a.D, 256)), dim3(256), 0, s,
                           (const T *)x, (const T *)init, a, sq, (T *)fin);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_conv_backward(const void *x, const ConvArgs &a, const void *init, const Seqs &sq, const void *dout,
                                const void *dfinal, void *dx, float *dw, float *dbias, void *dinit, hipStream_t s)
{
    if (sq.T > 0 && sq.N > 0)
        hipLaunchKernelGGL(kda_conv_bwd_dx_kernel<T>, dim3(conv_blocks((int64_t)sq.T * a.D, 256)), dim3(256), 0, s,
                           (const T *)x, (const T *)init, a, sq, (const T *)dout, (const T *)dfinal, (T *)dx);
    if (dinit && sq.N > 0)
        hipLaunchKernelGGL(kda_conv_bwd_dinit_kernel<T>, dim3(conv_blocks((int64_t)sq.N * (a.width - 1) * a.D, 256)),
                           dim3(256), 0, s, (const T *)x, (const T *)init, a, sq, (const T *)dout, (const T *)dfinal,
                           (T *)dinit);
    hipLaunchKernelGGL(kda_conv_bwd_dw_kernel<T>, dim3((unsigned)((a.D + 63) / 64)), dim3(64), 0, s, (const T *)x,
                       (const T *)init, a, sq, (const T *)dout, dw, dbias);
    return hipGetLastError();
}

}  // namespace kda

using namespace kda;

hipError_t kda_launch_conv(bool bf16, const void *x, const float *w, const float *bias, const void *init,
                           const int32_t *cu, int32_t N, int32_t T, int32_t D, int32_t width, bool silu, void *out,
                           void *fin, hipStream_t s)
{
    const ConvArgs a{w, bias, D, width, silu};
    const Seqs sq{cu, N, T};
    return bf16 ? launch_conv<bf16_t>(x, a, init, sq, out, fin, s) : launch_conv<float>(x, a, init, sq, out, fin, s);
}

hipError_t kda_launch_conv_step(bool bf16, const void *x, const float *w, const float *bias, void *state, int32_t N,
                                int32_t D, int32_t width, bool silu, void *out, hipStream_t s)
{
    const ConvArgs a{w, bias, D, width, silu};
    const unsigned blocks = conv_blocks((int64_t)N * D, 256);
    if (bf16)
        hipLaunchKernelGGL(kda_conv_step_kernel<bf16_t>, dim3(blocks), dim3(256), 0, s, (const bf16_t *)x,
                           (bf16_t *)state, a, N, (bf16_t *)out);
    else
        hipLaunchKernelGGL(kda_conv_step_kernel<float>, dim3(blocks), dim3(256), 0, s, (const float *)x,
                           (float *)state, a, N, (float *)out);
    return hipGetLastError();
}

size_t kda_conv_bwd_ws_bytes(int32_t, int32_t, int32_t, bool) { return 0; }

hipError_t kda_launch_conv_backward(bool bf16, const void *x, const float *w, const float *bias, const void *init,
                                    const int32_t *cu, int32_t N, int32_t T, int32_t D, int32_t width, bool silu,
                                    const void *dout, const void *dfinal, void *dx, float *dw, float *dbias,
                                    void *dinit, void *, hipStream_t s)
{
    const ConvArgs a{w, bias, D, width, silu};
    const Seqs sq{cu, N, T};
    return bf16 ? launch_conv_backward<bf16_t>(x, a, init, sq, dout, dfinal, dx, dw, dbias, dinit, s)
                : launch_conv_backward<float>(x, a, init, sq, dout, dfinal, dx, dw, dbias, dinit, s);
}

// kda_scan.hip -- the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per
// channel over packed sequences, its decode step and its gradients.
//
// One thread per (sequence, channel) walks its tokens.
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_seq.hpp"

namespace kda {

constexpr int TILE = 128;   // tokens between checkpoints

// out: h; chk: the state entering every TILE-th token; carried: exp(g_t) h_{t-1}
template <typename T>
__global__ void kda_scan_kernel(const T *x, const float *g, const float *init, Seqs sq, int64_t D, T *out, float *fin,
                                float *chk, float *carried)
{
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (id >= sq.N * D) return;
    const int32_t n = (int32_t)(id / D);
    const int64_t c = id % D;
    const int32_t t0 = sq.at(n), t1 = sq.at(n + 1);
    float h = init ? init[id] : 0.f;
    for (int32_t t = t0; t < t1; ++t) {
        const int64_t i = t * D + c;
        if (chk && t % TILE == 0) chk[(int64_t)(t / TILE) * D + c] = h;
        const float p = expf(g[i]) * h;
        if (carried) carried[i] = p;
        h = p + to_f(x[i]);
        if (out) out[i] = from_f<T>(h);
    }
    if (fin) fin[id] = h;
}

template <typename T>
__global__ void kda_scan_step_kernel(const T *x, const float *g, float *state, int64_t n, T *out)
{
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const float h = expf(g[i]) * state[i] + to_f(x[i]);
        state[i] = h;
        out[i] = from_f<T>(h);
    }
}

template <typename T>
__global__ void kda_scan_bwd_kernel(const float *g, Seqs sq, int64_t D, const T *dout, const float *dfinal,
                                    const float *carried, T *dx, float *dg, float *dinit)
{
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (id >= sq.N * D) return;
    const int32_t n = (int32_t)(id / D);
    const int64_t c = id % D;
    const int32_t t0 = sq.at(n), t1 = sq.at(n + 1);
    float e = dfinal ? dfinal[id] : 0.f;   // gradient of the state that leaves the token
    for (int32_t t = t1 - 1; t >= t0; --t) {
        const int64_t i = t * D + c;
        const float dh = to_f(dout[i]) + e;
        dx[i] = from_f<T>(dh);
        dg[i] = dh * carried[i];
        e = expf(g[i]) * dh;
    }
    if (dinit) dinit[id] = e;
}

inline unsigned blocks_of(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace kda

using namespace kda;

size_t kda_scan_ws_bytes(int32_t, int32_t) { return 0; }

hipError_t kda_launch_scan(bool bf16, const void *x, const float *g, const float *init, const int32_t *cu, int32_t N,
                           int32_t T, int32_t D, void *out, float *fin, float *chk, void *, hipStream_t s)
{
    const Seqs sq{cu, N, T};
    const unsigned blocks = blocks_of((int64_t)N * D, 64);
    if (bf16)
        hipLaunchKernelGGL(kda_scan_kernel<bf16_t>, dim3(blocks), dim3(64), 0, s, (const bf16_t *)x, g, init, sq,
                           (int64_t)D, (bf16_t *)out, fin, chk, (float *)nullptr);
    else
        hipLaunchKernelGGL(kda_scan_kernel<float>, dim3(blocks), dim3(64), 0, s, (const float *)x, g, init, sq,
                           (int64_t)D, (float *)out, fin, chk, (float *)nullptr);
    return hipGetLastError();
}

hipError_t kda_launch_scan_step(bool bf16, const void *x, const float *g, float *state, int64_t n, void *out,
                                hipStream_t s)
{
    const unsigned blocks = blocks_of(n, 256) < 65536 ? blocks_of(n, 256) : 65536;
    if (bf16)
        hipLaunchKernelGGL(kda_scan_step_kernel<bf16_t>, dim3(blocks), dim3(256), 0, s, (const bf16_t *)x, g, state, n,
                           (bf16_t *)out);
    else
        hipLaunchKernelGGL(kda_scan_step_kernel<float>, dim3(blocks), dim3(256), 0, s, (const float *)x, g, state, n,
                           (float *)out);
    return hipGetLastError();
}

size_t kda_scan_bwd_ws_bytes(int32_t T, int32_t D, bool) { return (size_t)T * D * sizeof(float); }

hipError_t kda_launch_scan_backward(bool bf16, const void *x, const float *g, const float *init, const int32_t *cu,
                                    int32_t N, int32_t T, int32_t D, const void *dout, const float *dfinal,
                                    const float *, void *dx, float *dg, float *dinit, void *ws, hipStream_t s)
{
    const Seqs sq{cu, N, T};
    const unsigned blocks = blocks_of((int64_t)N * D, 64);
    float *carried = (float *)ws;
    if (bf16) {
        hipLaunchKernelGGL(kda_scan_kernel<bf16_t>, dim3(blocks), dim3(64), 0, s, (const bf16_t *)x, g, init, sq,
                           (int64_t)D, (bf16_t *)nullptr, (float *)nullptr, (float *)nullptr, carried);
        hipLaunchKernelGGL(kda_scan_bwd_kernel<bf16_t>, dim3(blocks), dim3(64), 0, s, g, sq, (int64_t)D,
                           (const bf16_t *)dout, dfinal, carried, (bf16_t *)dx, dg, dinit);
    } else {
        hipLaunchKernelGGL(kda_scan_kernel<float>, dim3(blocks), dim3(64), 0, s, (const float *)x, g, init, sq,
                           (int64_t)D, (float *)nullptr, (float *)nullptr, (float *)nullptr, carried);
        hipLaunchKernelGGL(kda_scan_bwd_kernel<float>, dim3(blocks), dim3(64), 0, s, g, sq, (int64_t)D,
                           (const float *)dout, dfinal, carried, (float *)dx, dg, dinit);
    }
    return hipGetLastError();
}

// kda_layer.hpp -- launchers of the layer operators' kernels, as the host API
// calls them (kda_scan.hip, kda_conv.hip, kda_norm.hip).  Arguments have been
// checked; every launcher returns the HIP status of its launches.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

constexpr int32_t kMaxNormChannels = 16384;

// Channels of a column of work: 64 lanes of V, or a little less where the last
// column would otherwise be narrower than a lane (D >= V).  A lane that reaches
// past the last channel is moved back over its neighbour's; that neighbour is
// then in the same column, so that no two columns touch one channel's state.
inline int32_t kda_column_width(int32_t D, int V)
{
    int32_t w = 64 * V;
    while (w > V && (D - 1) % w + 1 < V) w -= V;
    return w;
}

// A launch counts its threads in 32 bits.  The ..._fits functions say whether the
// grid of a launcher, for the same arguments, has no more: the callers ask them.
inline bool kda_grid_ok(int64_t blocks, int threads) { return blocks <= (int64_t)UINT32_MAX / threads; }

bool kda_scan_fits(int32_t N, int32_t T, int32_t D);
size_t kda_scan_ws_bytes(int32_t T, int32_t D);
hipError_t kda_launch_scan(bool bf16, const void *x, const float *g, const float *init, const int32_t *cu, int32_t N,
                           int32_t T, int32_t D, void *out, float *fin, float *checkpoints, void *ws, hipStream_t s);
hipError_t kda_launch_scan_step(bool bf16, const void *x, const float *g, float *state, int64_t n, void *out,
                                hipStream_t s);
size_t kda_scan_bwd_ws_bytes(int32_t T, int32_t D, bool has_checkpoints);
hipError_t kda_launch_scan_backward(bool bf16, const void *x, const float *g, const float *init, const int32_t *cu,
                                    int32_t N, int32_t T, int32_t D, const void *dout, const float *dfinal,
                                    const float *checkpoints, void *dx, float *dg, float *dinit, void *ws,
                                    hipStream_t s);

bool kda_conv_fits(int32_t N, int32_t T, int32_t D, const void *init, const void *fin);
hipError_t kda_launch_conv(bool bf16, const void *x, const float *w, const float *bias, const void *init,
                           const int32_t *cu, int32_t N, int32_t T, int32_t D, int32_t width, bool silu, void *out,
                           void *fin, hipStream_t s);
bool kda_conv_step_fits(bool bf16, int32_t N, int32_t D);
hipError_t kda_launch_conv_step(bool bf16, const void *x, const float *w, const float *bias, void *state, int32_t N,
                                int32_t D, int32_t width, bool silu, void *out, hipStream_t s);
size_t kda_conv_bwd_ws_bytes(int32_t T, int32_t D, int32_t width, bool bf16);
bool kda_conv_backward_fits(int32_t N, int32_t T, int32_t D, int32_t width, const void *dfinal, const void *dinit);
hipError_t kda_launch_conv_backward(bool bf16, const void *x, const float *w, const float *bias, const void *init,
                                    const int32_t *cu, int32_t N, int32_t T, int32_t D, int32_t width, bool silu,
                                    const void *dout, const void *dfinal, void *dx, float *dw, float *dbias,
                                    void *dinit, void *ws, hipStream_t s);

bool kda_rmsnorm_fits(bool bf16, int32_t rows, int32_t D);
hipError_t kda_launch_rmsnorm(bool bf16, const void *x, const void *residual, const float *w, int32_t rows, int32_t D,
                              float eps, void *sum, void *out, uint8_t *mx, uint8_t *scales, hipStream_t s);
size_t kda_rmsnorm_bwd_ws_bytes(int32_t rows, int32_t D);
hipError_t kda_launch_rmsnorm_backward(bool bf16, const void *x, const float *w, const void *dout, const void *dres,
                                       int32_t rows, int32_t D, float eps, void *dx, float *dw, void *ws,
                                       hipStream_t s);

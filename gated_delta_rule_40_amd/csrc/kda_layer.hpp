// kda_layer.hpp -- launchers of the layer operators' kernels, as the host API
// calls them (kda_scan.hip, kda_conv.hip, kda_norm.hip, kda_qknorm.hip,
// kda_cache.hip, kda_cached_decode.hip, kda_verify.hip).  Arguments have been
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

// What kda_qknorm and its gradients share (include/kda.h); without a rotation rot is 0.
struct KdaQkNorm {
    const void *q, *k;
    int64_t q_stride, k_stride;
    const float *q_weight, *k_weight;
    const int32_t *positions;
    const float *inv_freq;
    const int32_t *pair_axis;
    int32_t tokens, q_heads, k_heads, dim, rot, axes;
    bool interleaved;
    int32_t norm;
    float eps, q_scale;
};
bool kda_qknorm_fits(bool bf16, const KdaQkNorm &a, bool back);
hipError_t kda_launch_qknorm(bool bf16, const KdaQkNorm &a, void *q_out, void *k_out, hipStream_t s);
size_t kda_qknorm_bwd_ws_bytes(int32_t d);
hipError_t kda_launch_qknorm_backward(bool bf16, bool grad_bf16, const KdaQkNorm &a, const void *dq_out, const void *dk_out,
                                      int64_t dq_stride, int64_t dk_stride, void *dq, void *dk, float *dq_weight,
                                      float *dk_weight, void *ws, hipStream_t s);

bool kda_cache_fits(bool bf16, int32_t entries, int32_t elems);
hipError_t kda_launch_cache_store(bool bf16, const void *src, const int32_t *slots, int32_t entries, int32_t elems,
                                  int format, int64_t entry_bytes, int32_t num_slots, uint8_t *cache, uint8_t *scales,
                                  hipStream_t s);
hipError_t kda_launch_cache_load(bool bf16, const uint8_t *cache, const uint8_t *scales, const int32_t *slots,
                                 int32_t entries, int32_t elems, int format, int64_t entry_bytes, int32_t num_slots,
                                 void *dst, hipStream_t s);
bool kda_cached_tokens_fits(int32_t N, int32_t H);
hipError_t kda_launch_cached_tokens(bool bf16, const void *q, const void *k, const void *v, const float *g, const float *beta,
                                    const int32_t *cu, const int32_t *num_tokens, uint8_t *cache, uint8_t *scales,
                                    const int32_t *slots, bool write, int32_t num_slots, int32_t N, int32_t T_tot,
                                    int32_t H, int format, void *out, hipStream_t s);

bool kda_verify_fits(int32_t N, int32_t vocab);
size_t kda_verify_ws_bytes(int32_t N, int32_t vocab);
hipError_t kda_launch_verify(bool bf16, const void *target, const void *draft, const int32_t *tokens, const int32_t *cu,
                             const float *accept_rand, const float *sample_rand, int32_t N, int32_t T_tot, int32_t vocab,
                             int32_t *num_tokens, int32_t *next_token, void *ws, hipStream_t s);

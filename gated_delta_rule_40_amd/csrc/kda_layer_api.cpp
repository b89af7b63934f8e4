// kda_layer_api.cpp -- host side of the layer operators of the libkda C ABI
// (kda_scan_*, kda_conv_*, kda_rmsnorm*, kda_qknorm*; declared in include/kda.h).
//
// Validates every argument before touching HIP and launches on the caller's
// stream.  Nothing is allocated and no stream is synchronised.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kda.h"
#include "kda_host.hpp"
#include "kda_layer.hpp"

using namespace kda_host;

namespace {

size_t checkpoint_bytes(int32_t T, int32_t D)
{
    return ((size_t)T + KDA_SCAN_TILE - 1) / KDA_SCAN_TILE * D * sizeof(float);
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- gated linear recurrence
size_t kda_scan_workspace_size(int32_t num_seqs, int32_t total_tokens, int32_t channels, kda_dtype dtype)
{
    if (num_seqs < 0 || total_tokens < 0 || channels <= 0 || !dtype_ok(dtype)) return 0;
    return kda_scan_ws_bytes(total_tokens, channels);
}

kda_status kda_scan_prefill(const void *x, const float *g, const float *initial_state,
                            const int32_t *cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                            int32_t channels, kda_dtype dtype, void *out, float *final_state,
                            float *checkpoints, void *workspace, size_t workspace_bytes,
                            kda_stream_t stream)
{
    if (!packed_ok(cu_seqlens, num_seqs, total_tokens, channels, dtype)) return KDA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)total_tokens * channels;
    if (!array_ok(x, n, elem_size(dtype)) || !array_ok(g, n, 4) || !array_ok(out, n, elem_size(dtype)) ||
        !aligned(initial_state, 4) || !aligned(final_state, 4) || !aligned(checkpoints, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t need = kda_scan_ws_bytes(total_tokens, channels);
    if (!workspace_ok(workspace, workspace_bytes, need, 8)) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0) return KDA_OK;
    if (!kda_scan_fits(num_seqs, total_tokens, channels)) return KDA_ERR_UNSUPPORTED;
    const size_t tokens = n * elem_size(dtype), state = (size_t)num_seqs * channels * 4;
    if (!keep_apart({{out, tokens, 1}, {final_state, state, 4}, {checkpoints, checkpoint_bytes(total_tokens, channels)},
                     {workspace, need}},
                    {{x, tokens}, {g, (size_t)n * 4}, {initial_state, state}, {cu_seqlens, cu_bytes(num_seqs)}}))
        return KDA_ERR_INVALID_ARG;
    if (kda_status v = check_cu(cu_seqlens, num_seqs, total_tokens, stream)) return v;
    return from_hip(kda_launch_scan(dtype == KDA_BF16, x, g, initial_state, cu_seqlens, num_seqs, total_tokens,
                                    channels, out, final_state, checkpoints, workspace, hip_stream(stream)));
}

kda_status kda_scan_decode_step(const void *x, const float *g, float *state_inout, int32_t num_seqs,
                                int32_t channels, kda_dtype dtype, void *out, kda_stream_t stream)
{
    if (!dtype_ok(dtype) || num_seqs < 0 || channels <= 0) return KDA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)num_seqs * channels;
    const size_t e = elem_size(dtype);
    if (!array_ok(x, n, e) || !array_ok(g, n, 4) || !array_ok(state_inout, n, 4) || !array_ok(out, n, e))
        return KDA_ERR_INVALID_ARG;
    if (n == 0) return KDA_OK;
    if (!keep_apart({{out, n * e, 1}, {state_inout, (size_t)n * 4}}, {{x, n * e}, {g, (size_t)n * 4}}))
        return KDA_ERR_INVALID_ARG;
    return from_hip(kda_launch_scan_step(dtype == KDA_BF16, x, g, state_inout, n, out, hip_stream(stream)));
}

size_t kda_scan_backward_workspace_size(int32_t num_seqs, int32_t total_tokens, int32_t channels,
                                        kda_dtype dtype, int32_t has_checkpoints)
{
    if (num_seqs < 0 || total_tokens < 0 || channels <= 0 || !dtype_ok(dtype)) return 0;
    return kda_scan_bwd_ws_bytes(total_tokens, channels, has_checkpoints != 0);
}

kda_status kda_scan_backward(const void *x, const float *g, const float *initial_state,
                             const int32_t *cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                             int32_t channels, kda_dtype dtype, const void *dout, const float *dfinal,
                             const float *checkpoints, void *dx, float *dg, float *dinit,
                             void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    if (!packed_ok(cu_seqlens, num_seqs, total_tokens, channels, dtype)) return KDA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)total_tokens * channels;
    const size_t e = elem_size(dtype);
    if (!array_ok(x, n, e) || !array_ok(g, n, 4) || !array_ok(dout, n, e) || !array_ok(dx, n, e) ||
        !array_ok(dg, n, 4) || !aligned(initial_state, 4) || !aligned(dfinal, 4) || !aligned(checkpoints, 4) ||
        !aligned(dinit, 4))
        return KDA_ERR_INVALID_ARG;
    const size_t need = kda_scan_bwd_ws_bytes(total_tokens, channels, checkpoints != nullptr);
    if (!workspace_ok(workspace, workspace_bytes, need, 8)) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0) return KDA_OK;
    if (!kda_scan_fits(num_seqs, total_tokens, channels)) return KDA_ERR_UNSUPPORTED;
    const size_t tokens = n * e, gates = (size_t)n * 4, state = (size_t)num_seqs * channels * 4;
    if (!keep_apart({{dx, tokens, 1 | 2}, {dg, gates, 4}, {dinit, state}, {workspace, need}},
                    {{x, tokens}, {dout, tokens}, {g, gates}, {initial_state, state}, {dfinal, state},
                     {cu_seqlens, cu_bytes(num_seqs)}, {checkpoints, checkpoint_bytes(total_tokens, channels)}}))
        return KDA_ERR_INVALID_ARG;
    if (kda_status v = check_cu(cu_seqlens, num_seqs, total_tokens, stream)) return v;
    return from_hip(kda_launch_scan_backward(dtype == KDA_BF16, x, g, initial_state, cu_seqlens, num_seqs,
                                             total_tokens, channels, dout, dfinal, checkpoints, dx, dg, dinit,
                                             workspace, hip_stream(stream)));
}

// ---------------------------------------------------------------- short causal convolution
kda_status kda_conv_prefill(const void *x, const float *weight, const float *bias, const void *initial_state,
                            const int32_t *cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                            int32_t channels, int32_t width, int32_t silu, kda_dtype dtype, void *out,
                            void *final_state, kda_stream_t stream)
{
    if (!packed_ok(cu_seqlens, num_seqs, total_tokens, channels, dtype) || width <= 0) return KDA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)total_tokens * channels;
    const size_t e = elem_size(dtype);
    if (!array_ok(x, n, e) || !array_ok(out, n, e) || !weight || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(initial_state, e) || !aligned(final_state, e))
        return KDA_ERR_INVALID_ARG;
    if (width < 2 || width > 4) return KDA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return KDA_OK;
    if (!kda_conv_fits(num_seqs, total_tokens, channels, initial_state, final_state)) return KDA_ERR_UNSUPPORTED;
    const size_t state = (size_t)num_seqs * (width - 1) * channels * e;
    if (!keep_apart({{out, n * e}, {final_state, state, 1}},
                    {{initial_state, state}, {x, n * e}, {weight, (size_t)channels * width * 4},
                     {bias, (size_t)channels * 4}, {cu_seqlens, cu_bytes(num_seqs)}}))
        return KDA_ERR_INVALID_ARG;
    if (kda_status v = check_cu(cu_seqlens, num_seqs, total_tokens, stream)) return v;
    return from_hip(kda_launch_conv(dtype == KDA_BF16, x, weight, bias, initial_state, cu_seqlens, num_seqs,
                                    total_tokens, channels, width, silu != 0, out, final_state,
                                    hip_stream(stream)));
}

kda_status kda_conv_decode_step(const void *x, const float *weight, const float *bias, void *state_inout,
                                int32_t num_seqs, int32_t channels, int32_t width, int32_t silu,
                                kda_dtype dtype, void *out, kda_stream_t stream)
{
    if (!dtype_ok(dtype) || num_seqs < 0 || channels <= 0 || width <= 0) return KDA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)num_seqs * channels;
    const size_t e = elem_size(dtype);
    if (!array_ok(x, n, e) || !array_ok(out, n, e) || !array_ok(state_inout, n, e) || !weight ||
        !aligned(weight, 4) || !aligned(bias, 4))
        return KDA_ERR_INVALID_ARG;
    if (width < 2 || width > 4) return KDA_ERR_UNSUPPORTED;
    if (n == 0) return KDA_OK;
    if (!kda_conv_step_fits(dtype == KDA_BF16, num_seqs, channels)) return KDA_ERR_UNSUPPORTED;
    if (!keep_apart({{out, n * e, 1}, {state_inout, n * (width - 1) * e}},
                    {{x, n * e}, {weight, (size_t)channels * width * 4}, {bias, (size_t)channels * 4}}))
        return KDA_ERR_INVALID_ARG;
    return from_hip(kda_launch_conv_step(dtype == KDA_BF16, x, weight, bias, state_inout, num_seqs, channels, width,
                                         silu != 0, out, hip_stream(stream)));
}

size_t kda_conv_backward_workspace_size(int32_t num_seqs, int32_t total_tokens, int32_t channels,
                                        int32_t width, kda_dtype dtype)
{
    if (num_seqs < 0 || total_tokens < 0 || channels <= 0 || width < 2 || width > 4 || !dtype_ok(dtype)) return 0;
    return kda_conv_bwd_ws_bytes(total_tokens, channels, width, dtype == KDA_BF16);
}

kda_status kda_conv_backward(const void *x, const float *weight, const float *bias, const void *initial_state,
                             const int32_t *cu_seqlens, int32_t num_seqs, int32_t total_tokens,
                             int32_t channels, int32_t width, int32_t silu, kda_dtype dtype,
                             const void *dout, const void *dfinal, void *dx, float *dweight, float *dbias,
                             void *dinit, void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    if (!packed_ok(cu_seqlens, num_seqs, total_tokens, channels, dtype) || width <= 0) return KDA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)total_tokens * channels;
    const size_t e = elem_size(dtype);
    if (!array_ok(x, n, e) || !array_ok(dout, n, e) || !array_ok(dx, n, e) || !weight || !dweight ||
        !aligned(weight, 4) || !aligned(bias, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) ||
        !aligned(initial_state, e) || !aligned(dfinal, e) || !aligned(dinit, e))
        return KDA_ERR_INVALID_ARG;
    if (width < 2 || width > 4) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda_conv_bwd_ws_bytes(total_tokens, channels, width, dtype == KDA_BF16);
    if (!workspace_ok(workspace, workspace_bytes, need, 4)) return KDA_ERR_INVALID_ARG;
    if (!kda_conv_backward_fits(num_seqs, total_tokens, channels, width, dfinal, dinit)) return KDA_ERR_UNSUPPORTED;
    const size_t state = (size_t)num_seqs * (width - 1) * channels * e, row = (size_t)channels * 4;
    if (!keep_apart({{dx, n * e}, {dweight, row * width}, {dbias, row}, {dinit, state}, {workspace, need}},
                    {{x, n * e}, {dout, n * e}, {weight, row * width}, {bias, row}, {initial_state, state},
                     {dfinal, state}, {cu_seqlens, cu_bytes(num_seqs)}}))
        return KDA_ERR_INVALID_ARG;
    if (num_seqs > 0)
        if (kda_status v = check_cu(cu_seqlens, num_seqs, total_tokens, stream)) return v;
    // without sequences the weights' gradients are still written (zeros)
    return from_hip(kda_launch_conv_backward(dtype == KDA_BF16, x, weight, bias, initial_state, cu_seqlens, num_seqs,
                                             total_tokens, channels, width, silu != 0, dout, dfinal, dx, dweight,
                                             dbias, dinit, workspace, hip_stream(stream)));
}

// ---------------------------------------------------------------- residual and norm
kda_status kda_rmsnorm(const void *x, const void *residual, const float *weight, int32_t rows,
                       int32_t channels, float eps, kda_dtype dtype, void *residual_out, void *out,
                       uint8_t *out_mx, uint8_t *scales, kda_stream_t stream)
{
    if (!dtype_ok(dtype) || rows < 0 || channels <= 0 || !std::isfinite(eps) || eps < 0.f) return KDA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)rows * channels;
    const size_t e = elem_size(dtype);
    if (!array_ok(x, n, e) || !aligned(residual, e) || !aligned(weight, 4) || !aligned(residual_out, e) ||
        !aligned(out, e))
        return KDA_ERR_INVALID_ARG;
    if (n && ((residual_out && !residual) || (out_mx != nullptr) != (scales != nullptr) || (!out && !out_mx)))
        return KDA_ERR_INVALID_ARG;
    if (channels > kMaxNormChannels) return KDA_ERR_UNSUPPORTED;
    if (n == 0) return KDA_OK;
    if (!kda_rmsnorm_fits(dtype == KDA_BF16, rows, channels)) return KDA_ERR_UNSUPPORTED;
    if (!keep_apart({{residual_out, n * e, 1 | 2}, {out, n * e, 1 | 2}, {out_mx, (size_t)n},
                     {scales, (size_t)rows * ((channels + KDA_MX_BLOCK - 1) / KDA_MX_BLOCK)}},
                    {{x, n * e}, {residual, n * e}, {weight, (size_t)channels * 4}}))
        return KDA_ERR_INVALID_ARG;
    return from_hip(kda_launch_rmsnorm(dtype == KDA_BF16, x, residual, weight, rows, channels, eps, residual_out, out,
                                       out_mx, scales, hip_stream(stream)));
}

size_t kda_rmsnorm_backward_workspace_size(int32_t rows, int32_t channels, kda_dtype dtype)
{
    if (rows < 0 || channels <= 0 || channels > kMaxNormChannels || !dtype_ok(dtype)) return 0;
    return kda_rmsnorm_bwd_ws_bytes(rows, channels);
}

kda_status kda_rmsnorm_backward(const void *x, const float *weight, const void *dout, const void *dresidual,
                                int32_t rows, int32_t channels, float eps, kda_dtype dtype, void *dx,
                                float *dweight, void *workspace, size_t workspace_bytes,
                                kda_stream_t stream)
{
    if (!dtype_ok(dtype) || rows < 0 || channels <= 0 || !std::isfinite(eps) || eps < 0.f) return KDA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)rows * channels;
    const size_t e = elem_size(dtype);
    if (!array_ok(x, n, e) || !array_ok(dout, n, e) || !array_ok(dx, n, e) || !aligned(dresidual, e) ||
        !aligned(weight, 4) || !aligned(dweight, 4))
        return KDA_ERR_INVALID_ARG;
    if (channels > kMaxNormChannels) return KDA_ERR_UNSUPPORTED;
    const size_t need = dweight ? kda_rmsnorm_bwd_ws_bytes(rows, channels) : 0, row = (size_t)channels * 4;
    if (!workspace_ok(workspace, workspace_bytes, need, 4)) return KDA_ERR_INVALID_ARG;
    if (n == 0 && !dweight) return KDA_OK;
    if (!keep_apart({{dx, n * e, 1 | 2 | 4}, {dweight, row}, {workspace, need}},
                    {{x, n * e}, {dout, n * e}, {dresidual, n * e}, {weight, row}}))
        return KDA_ERR_INVALID_ARG;
    return from_hip(kda_launch_rmsnorm_backward(dtype == KDA_BF16, x, weight, dout, dresidual, rows, channels, eps,
                                                dx, dweight, workspace, hip_stream(stream)));
}

// ---------------------------------------------------------------- norm and rotation of queries and keys
namespace {

constexpr int64_t kMaxStride = INT64_C(1) << 29;   // elements between tokens: spans stay below 2^62 bytes

// What forward and backward check alike.
kda_status check_qknorm(const KdaQkNorm &a, kda_dtype dtype, bool in_use)
{
    if (!dtype_ok(dtype) || a.tokens < 0 || a.q_heads < 0 || a.k_heads < 0 || a.dim <= 0 || a.rot < 0 || a.rot > a.dim ||
        a.rot % 2 || a.norm < KDA_NORM_NONE || a.norm > KDA_NORM_RMS || !std::isfinite(a.eps) || a.eps < 0.f ||
        !std::isfinite(a.q_scale))
        return KDA_ERR_INVALID_ARG;
    const size_t e = elem_size(dtype);
    const int64_t qc = (int64_t)a.q_heads * a.dim, kc = (int64_t)a.k_heads * a.dim;
    if (qc > INT32_MAX - 65536 || kc > INT32_MAX - 65536) return KDA_ERR_INVALID_ARG;
    if (!array_ok(a.q, a.tokens * qc, e) || !array_ok(a.k, a.tokens * kc, e) || (a.tokens > 0 && (a.q_stride < qc || a.k_stride < kc)) ||
        !aligned(a.q_weight, 4) || !aligned(a.k_weight, 4))
        return KDA_ERR_INVALID_ARG;
    if (a.q_stride > kMaxStride || a.k_stride > kMaxStride) return KDA_ERR_INVALID_ARG;
    if (a.rot && in_use &&
        (a.axes <= 0 || !a.positions || !aligned(a.positions, 4) || !a.inv_freq || !aligned(a.inv_freq, 4) || !aligned(a.pair_axis, 4)))
        return KDA_ERR_INVALID_ARG;
    return a.dim > KDA_QKNORM_MAX_DIM ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

// the arrays that are read: q, k, weights, positions, frequencies, axes
constexpr int kQkInputs = 7;
void qknorm_inputs(const KdaQkNorm &a, size_t e, Rows (&in)[kQkInputs])
{
    const int64_t n = a.tokens, qw = (int64_t)a.q_heads * a.dim * e, kw = (int64_t)a.k_heads * a.dim * e;
    in[0] = {a.q, n, qw, (int64_t)(a.q_stride * e)};
    in[1] = {a.k, n, kw, (int64_t)(a.k_stride * e)};
    in[2] = dense(a.q_weight, (size_t)a.dim * 4), in[3] = dense(a.k_weight, (size_t)a.dim * 4);
    const size_t pairs = a.rot / 2;
    in[4] = dense(a.rot ? a.positions : nullptr, (size_t)a.axes * n * 4);
    in[5] = dense(a.rot ? a.inv_freq : nullptr, pairs * 4), in[6] = dense(a.rot ? a.pair_axis : nullptr, pairs * 4);
}

// Whether `o` shares memory with one of `in`, other than lying whole in the place of number `may`.
bool meets_any(const Rows &o, const Rows *in, int n, int may)
{
    for (int i = 0; i < n; ++i) {
        const bool same = i == may && o.p == in[i].p && (o.rows <= 1 || o.pitch == in[i].pitch);
        if (!same && rows_meet(o, in[i])) return true;
    }
    return false;
}

}  // namespace

kda_status kda_qknorm(const void *q, const void *k, int64_t q_stride, int64_t k_stride, const float *q_weight,
                      const float *k_weight, const int32_t *positions, const float *inv_freq,
                      const int32_t *pair_axis, int32_t num_tokens, int32_t num_q_heads, int32_t num_k_heads,
                      int32_t head_dim, int32_t rot_dim, int32_t num_axes, int32_t interleaved, kda_norm norm,
                      float eps, float q_scale, kda_dtype dtype, void *q_out, void *k_out, kda_stream_t stream)
{
    const KdaQkNorm a{q, k, q_stride, k_stride, q_weight, k_weight, positions, inv_freq, pair_axis, num_tokens, num_q_heads,
                      num_k_heads, head_dim, rot_dim, num_axes, interleaved != 0, norm, eps, q_scale};
    const bool in_use = num_tokens > 0 && (num_q_heads > 0 || num_k_heads > 0);
    if (kda_status st = check_qknorm(a, dtype, in_use)) return st;
    const size_t e = elem_size(dtype);
    const int64_t qc = (int64_t)num_q_heads * head_dim, kc = (int64_t)num_k_heads * head_dim;
    if (!array_ok(q_out, num_tokens * qc, e) || !array_ok(k_out, num_tokens * kc, e)) return KDA_ERR_INVALID_ARG;
    if (!in_use) return KDA_OK;
    Rows in[kQkInputs];
    qknorm_inputs(a, e, in);
    const Rows qo{q_out, num_tokens, (int64_t)(qc * e), (int64_t)(qc * e)}, ko{k_out, num_tokens, (int64_t)(kc * e), (int64_t)(kc * e)};
    if (rows_meet(qo, ko) || meets_any(qo, in, kQkInputs, 0) || meets_any(ko, in, kQkInputs, 1)) return KDA_ERR_INVALID_ARG;
    if (!kda_qknorm_fits(dtype == KDA_BF16, a, false)) return KDA_ERR_UNSUPPORTED;
    return from_hip(kda_launch_qknorm(dtype == KDA_BF16, a, q_out, k_out, hip_stream(stream)));
}

size_t kda_qknorm_backward_workspace_size(int32_t num_tokens, int32_t num_q_heads, int32_t num_k_heads,
                                          int32_t head_dim, kda_dtype dtype)
{
    if (num_tokens < 0 || num_q_heads < 0 || num_k_heads < 0 || head_dim <= 0 || head_dim > KDA_QKNORM_MAX_DIM || !dtype_ok(dtype))
        return 0;
    return kda_qknorm_bwd_ws_bytes(head_dim);
}

kda_status kda_qknorm_backward(const void *q, const void *k, int64_t q_stride, int64_t k_stride,
                               const float *q_weight, const float *k_weight, const int32_t *positions,
                               const float *inv_freq, const int32_t *pair_axis, int32_t num_tokens,
                               int32_t num_q_heads, int32_t num_k_heads, int32_t head_dim, int32_t rot_dim,
                               int32_t num_axes, int32_t interleaved, kda_norm norm, float eps, float q_scale,
                               kda_dtype dtype, kda_dtype grad_dtype, const void *dq_out, const void *dk_out,
                               int64_t dq_stride, int64_t dk_stride, void *dq, void *dk, float *dq_weight,
                               float *dk_weight, void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    const KdaQkNorm a{q, k, q_stride, k_stride, q_weight, k_weight, positions, inv_freq, pair_axis, num_tokens, num_q_heads,
                      num_k_heads, head_dim, rot_dim, num_axes, interleaved != 0, norm, eps, q_scale};
    const bool in_use = num_tokens > 0 && (num_q_heads > 0 || num_k_heads > 0);
    if (kda_status st = check_qknorm(a, dtype, in_use)) return st;
    if (!dtype_ok(grad_dtype) || (grad_dtype == KDA_BF16 && dtype != KDA_BF16)) return KDA_ERR_INVALID_ARG;
    const size_t e = elem_size(dtype), ge = elem_size(grad_dtype);
    const int64_t n = num_tokens, qc = (int64_t)num_q_heads * head_dim, kc = (int64_t)num_k_heads * head_dim;
    if (!array_ok(dq_out, n * qc, ge) || !array_ok(dk_out, n * kc, ge) || !array_ok(dq, n * qc, e) || !array_ok(dk, n * kc, e) ||
        (n > 0 && (dq_stride < qc || dk_stride < kc)) || dq_stride > kMaxStride || dk_stride > kMaxStride ||
        !aligned(dq_weight, 4) || !aligned(dk_weight, 4) || (dq_weight && !q_weight) || (dk_weight && !k_weight))
        return KDA_ERR_INVALID_ARG;
    const size_t need = dq_weight || dk_weight ? kda_qknorm_bwd_ws_bytes(head_dim) : 0;
    if (!workspace_ok(workspace, workspace_bytes, need, 4)) return KDA_ERR_INVALID_ARG;
    if (!in_use && !need) return KDA_OK;
    Rows in[kQkInputs + 2];
    {
        Rows first[kQkInputs];
        qknorm_inputs(a, e, first);
        std::copy(first, first + kQkInputs, in);
        in[kQkInputs] = dense(dq_out, n * qc * ge), in[kQkInputs + 1] = dense(dk_out, n * kc * ge);
    }
    const Rows outs[] = {{dq, n, (int64_t)(qc * e), (int64_t)(dq_stride * e)}, {dk, n, (int64_t)(kc * e), (int64_t)(dk_stride * e)},
                         dense(dq_weight, (size_t)head_dim * 4), dense(dk_weight, (size_t)head_dim * 4), dense(workspace, need)};
    for (int i = 0; i < 5; ++i) {
        if (meets_any(outs[i], in, kQkInputs + 2, i < 2 ? i : -1)) return KDA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (rows_meet(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
    }
    if (!kda_qknorm_fits(dtype == KDA_BF16, a, true)) return KDA_ERR_UNSUPPORTED;
    // without tokens the weights' gradients are still written (zeros)
    return from_hip(kda_launch_qknorm_backward(dtype == KDA_BF16, grad_dtype == KDA_BF16, a, dq_out, dk_out, dq_stride, dk_stride,
                                               dq, dk, dq_weight, dk_weight, workspace, hip_stream(stream)));
}

}  // extern "C"

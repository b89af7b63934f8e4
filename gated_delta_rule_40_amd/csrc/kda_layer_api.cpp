// kda_layer_api.cpp -- host side of the layer operators of the libkda C ABI
// (kda_scan_*, kda_conv_*, kda_rmsnorm*; declared in include/kda.h).
//
// Validates every argument before touching HIP and launches on the caller's
// stream.  Nothing is allocated and no stream is synchronised.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "kda.h"
#include "kda_host.hpp"
#include "kda_layer.hpp"

using namespace kda_host;

namespace {

bool dtype_ok(kda_dtype dtype) { return dtype == KDA_F32 || dtype == KDA_BF16; }
size_t elem_size(kda_dtype dtype) { return dtype == KDA_BF16 ? 2 : 4; }

// A token array: present (unless it has no elements) and aligned to its type.
bool array_ok(const void *p, int64_t elems, size_t size) { return (p || elems == 0) && aligned(p, size); }

// Arrays in bytes.  Bit i of an output's `may`: it may take the place of input i.
struct In {
    const void *p;
    size_t n;
};
struct Out {
    const void *p;
    size_t n;
    unsigned may;
};

template <typename A, typename B> bool meet(const A &a, const B &b)
{
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n && b.n && (p < q ? q - p < a.n : p - q < b.n);
}

// Whether no output shares memory with another one, or with an input that it is not, whole, in the place of.
bool keep_apart(std::initializer_list<Out> outs, std::initializer_list<In> ins)
{
    for (const Out *o = outs.begin(); o != outs.end(); ++o) {
        for (const Out *other = outs.begin(); other != o; ++other)
            if (meet(*o, *other)) return false;
        for (const In *i = ins.begin(); i != ins.end(); ++i)
            if (meet(*o, *i) && !(o->may >> (i - ins.begin()) & 1 && o->p == i->p)) return false;
    }
    return true;
}

kda_status from_hip(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH; }

hipStream_t hip_stream(kda_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

// What the packed calls share: sizes, type, cu_seqlens.  The kernels look a
// tile beyond a token, and a wave beyond a sequence, in int32.
bool packed_ok(const int32_t *cu, int32_t N, int32_t T, int32_t D, kda_dtype dtype)
{
    return dtype_ok(dtype) && N >= 0 && N <= INT32_MAX - 65536 && T >= 0 && T <= INT32_MAX - 65536 && D > 0 && cu &&
           aligned(cu, 4);
}

bool workspace_ok(const void *ws, size_t bytes, size_t need, size_t align)
{
    return need == 0 || (ws && aligned(ws, align) && bytes >= need);
}

size_t cu_bytes(int32_t N) { return ((size_t)N + 1) * sizeof(int32_t); }
size_t checkpoint_bytes(int32_t T, int32_t D)
{
    return ((size_t)T + KDA_SCAN_TILE - 1) / KDA_SCAN_TILE * D * sizeof(float);
}

kda_status check_cu(const int32_t *cu, int32_t N, int32_t T, kda_stream_t stream)
{
    return validate_enabled() ? validate_cu(cu, N, T, hip_stream(stream)) : KDA_OK;
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

}  // extern "C"

// kda_cache_api.cpp -- host side of the libkda C ABI's calls around cached states
// and drafted tokens (kda_cache_*, kda_decode_tokens_cached, kda_verify_drafts;
// declared in include/kda.h).
//
// Validates every argument before touching HIP and launches on the caller's
// stream.  Nothing is allocated and no stream is synchronised.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_host.hpp"
#include "kda_layer.hpp"

using namespace kda_host;

namespace {

constexpr int32_t kDim = 128;                        // dk = dv
constexpr int32_t kMaxVocab = INT32_C(1) << 30;

bool format_ok(kda_cache_format f) { return f == KDA_CACHE_FP8 || f == KDA_CACHE_INT8 || f == KDA_CACHE_FP4; }

size_t entry_scales(int64_t elems) { return (size_t)((elems + KDA_MX_BLOCK - 1) / KDA_MX_BLOCK); }

// What store and load check alike.
kda_status check_cache(const void *rows, const int32_t *slots, int32_t num_entries, int32_t entry_elems, kda_dtype dtype,
                       kda_cache_format format, int32_t num_slots, const uint8_t *cache, const uint8_t *scales)
{
    if (!dtype_ok(dtype) || !format_ok(format) || num_entries < 0 || entry_elems <= 0 || num_slots < 0) return KDA_ERR_INVALID_ARG;
    if (!array_ok(rows, num_entries, elem_size(dtype)) || !array_ok(slots, num_entries, 4) || !array_ok(cache, num_slots, 1) ||
        !array_ok(scales, num_slots, 1))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_cache_entry_bytes(int32_t entry_elems, kda_cache_format format)
{
    if (entry_elems < 0 || !format_ok(format)) return 0;
    return format == KDA_CACHE_FP4 ? ((size_t)entry_elems + 1) / 2 : (size_t)entry_elems;
}

kda_status kda_cache_store(const void *src, const int32_t *slots, int32_t num_entries, int32_t entry_elems,
                           kda_dtype dtype, kda_cache_format format, int32_t num_slots, uint8_t *cache,
                           uint8_t *scales, kda_stream_t stream)
{
    if (kda_status st = check_cache(src, slots, num_entries, entry_elems, dtype, format, num_slots, cache, scales)) return st;
    if (num_entries == 0 || num_slots == 0) return KDA_OK;
    const size_t bytes = kda_cache_entry_bytes(entry_elems, format);
    if (!kda_cache_fits(dtype == KDA_BF16, num_entries, entry_elems)) return KDA_ERR_UNSUPPORTED;
    if (!keep_apart({{cache, num_slots * bytes}, {scales, num_slots * entry_scales(entry_elems)}},
                    {{src, (size_t)num_entries * entry_elems * elem_size(dtype)}, {slots, (size_t)num_entries * 4}}))
        return KDA_ERR_INVALID_ARG;
    if (kda_status v = check_slots(slots, num_entries, num_slots, stream)) return v;
    return from_hip(kda_launch_cache_store(dtype == KDA_BF16, src, slots, num_entries, entry_elems, format, (int64_t)bytes,
                                           num_slots, cache, scales, hip_stream(stream)));
}

kda_status kda_cache_load(const uint8_t *cache, const uint8_t *scales, const int32_t *slots, int32_t num_entries,
                          int32_t entry_elems, kda_dtype dtype, kda_cache_format format, int32_t num_slots,
                          void *dst, kda_stream_t stream)
{
    if (kda_status st = check_cache(dst, slots, num_entries, entry_elems, dtype, format, num_slots, cache, scales)) return st;
    if (num_entries == 0) return KDA_OK;
    const size_t bytes = kda_cache_entry_bytes(entry_elems, format);
    if (!kda_cache_fits(dtype == KDA_BF16, num_entries, entry_elems)) return KDA_ERR_UNSUPPORTED;
    if (!keep_apart({{dst, (size_t)num_entries * entry_elems * elem_size(dtype)}},
                    {{cache, num_slots * bytes}, {scales, num_slots * entry_scales(entry_elems)}, {slots, (size_t)num_entries * 4}}))
        return KDA_ERR_INVALID_ARG;
    return from_hip(kda_launch_cache_load(dtype == KDA_BF16, cache, scales, slots, num_entries, entry_elems, format,
                                          (int64_t)bytes, num_slots, dst, hip_stream(stream)));
}

kda_status kda_decode_tokens_cached(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                    const int32_t *cu_seqlens, const int32_t *num_tokens, uint8_t *cache,
                                    uint8_t *scales, const int32_t *slots, int32_t write, int32_t num_slots,
                                    int32_t num_seqs, int32_t total_tokens, int32_t num_heads, int32_t dk,
                                    int32_t dv, kda_dtype dtype, kda_cache_format format, void *out,
                                    kda_stream_t stream)
{
    if (!format_ok(format) || num_heads <= 0 || dk <= 0 || dv <= 0 || num_slots < 0 ||
        !packed_ok(cu_seqlens, num_seqs, total_tokens, num_heads, dtype))
        return KDA_ERR_INVALID_ARG;
    const size_t e = elem_size(dtype);
    if (!array_ok(q, total_tokens, e) || !array_ok(k, total_tokens, e) || !array_ok(v, total_tokens, e) ||
        !array_ok(g, total_tokens, 4) || !array_ok(beta, total_tokens, 4) || !aligned(out, e) || !aligned(num_tokens, 4) ||
        !array_ok(slots, num_seqs, 4) || !array_ok(cache, num_slots, 1) || !array_ok(scales, num_slots, 1) ||
        (!out && !write && total_tokens > 0))
        return KDA_ERR_INVALID_ARG;
    if (dk != kDim || dv != kDim) return KDA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
    if (!kda_cached_tokens_fits(num_seqs, num_heads)) return KDA_ERR_UNSUPPORTED;
    const size_t rows = (size_t)total_tokens * num_heads, token = rows * kDim * e, state = (size_t)num_slots * num_heads * kDim;
    const Out o{out, token, 0};
    const In codes{cache, state * kda_cache_entry_bytes(kDim, format)}, scl{scales, state * entry_scales(kDim)};
    const std::initializer_list<In> ins = {{q, token}, {k, token}, {v, token}, {g, rows * kDim * 4}, {beta, rows * 4},
                                           {cu_seqlens, cu_bytes(num_seqs)}, {num_tokens, (size_t)num_seqs * 4},
                                           {slots, (size_t)num_seqs * 4}};
    if (!keep_apart({o}, ins) || !keep_apart({o}, {codes, scl}) ||
        (write && !keep_apart({{codes.p, codes.n}, {scl.p, scl.n}}, ins)))
        return KDA_ERR_INVALID_ARG;
    if (kda_status s = check_cu(cu_seqlens, num_seqs, total_tokens, stream)) return s;
    if (write)
        if (kda_status s = check_slots(slots, num_seqs, num_slots, stream)) return s;
    return from_hip(kda_launch_cached_tokens(dtype == KDA_BF16, q, k, v, g, beta, cu_seqlens, num_tokens, cache, scales, slots,
                                             write != 0, num_slots, num_seqs, total_tokens, num_heads, format, out,
                                             hip_stream(stream)));
}

size_t kda_verify_drafts_workspace_size(int32_t num_seqs, int32_t vocab, kda_dtype dtype)
{
    if (num_seqs < 0 || vocab <= 0 || vocab > kMaxVocab || !dtype_ok(dtype)) return 0;
    return kda_verify_ws_bytes(num_seqs, vocab);
}

kda_status kda_verify_drafts(const void *target_probs, const void *draft_probs, const int32_t *tokens,
                             const int32_t *cu_seqlens, const float *accept_rand, const float *sample_rand,
                             int32_t num_seqs, int32_t total_tokens, int32_t vocab, kda_dtype dtype,
                             int32_t *num_tokens, int32_t *next_token, void *workspace, size_t workspace_bytes,
                             kda_stream_t stream)
{
    if (!packed_ok(cu_seqlens, num_seqs, total_tokens, vocab, dtype)) return KDA_ERR_INVALID_ARG;
    const size_t e = elem_size(dtype);
    if (!array_ok(target_probs, total_tokens, e) || !aligned(draft_probs, e) || !array_ok(tokens, total_tokens, 4) ||
        !array_ok(accept_rand, total_tokens, 4) || !array_ok(sample_rand, num_seqs, 4) || !array_ok(num_tokens, num_seqs, 4) ||
        !array_ok(next_token, num_seqs, 4))
        return KDA_ERR_INVALID_ARG;
    if (vocab > kMaxVocab) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda_verify_ws_bytes(num_seqs, vocab);
    if (!workspace_ok(workspace, workspace_bytes, need, 8)) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0) return KDA_OK;
    if (!kda_verify_fits(num_seqs, vocab)) return KDA_ERR_UNSUPPORTED;
    const size_t probs = (size_t)total_tokens * vocab * e, seqs = (size_t)num_seqs * 4;
    if (!keep_apart({{num_tokens, seqs}, {next_token, seqs}, {workspace, need}},
                    {{target_probs, probs}, {draft_probs, probs}, {tokens, (size_t)total_tokens * 4},
                     {cu_seqlens, cu_bytes(num_seqs)}, {accept_rand, (size_t)total_tokens * 4}, {sample_rand, seqs}}))
        return KDA_ERR_INVALID_ARG;
    if (kda_status v = check_cu(cu_seqlens, num_seqs, total_tokens, stream)) return v;
    return from_hip(kda_launch_verify(dtype == KDA_BF16, target_probs, draft_probs, tokens, cu_seqlens, accept_rand, sample_rand,
                                      num_seqs, total_tokens, vocab, num_tokens, next_token, workspace, hip_stream(stream)));
}

}  // extern "C"

// kda_host.hpp -- host-side helpers shared by the C ABI's entry points:
// pointer alignment, the opt-in check of cu_seqlens, and the argument checks of
// the operators around the recurrence.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <memory>
#include <new>

#include "kda.h"

namespace kda_host {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// KDA_VALIDATE=1 in the environment (read once): the entry points that take
// cu_seqlens copy it to the host, synchronising `stream`, and check it before
// launching anything.  Off by default, since it costs a synchronisation.
inline bool validate_enabled()
{
    static std::atomic<int> state{-1};
    int v = state.load(std::memory_order_relaxed);
    if (v < 0) {
        const char *e = std::getenv("KDA_VALIDATE");
        v = (e && std::strcmp(e, "1") == 0) ? 1 : 0;
        state.store(v, std::memory_order_relaxed);
    }
    return v == 1;
}

// cu[0] = 0, non-decreasing, cu[N] <= T.  Returns KDA_ERR_INVALID_ARG for
// contents that break this, KDA_ERR_LAUNCH if the copy itself fails.
inline kda_status validate_cu(const int32_t *cu, int32_t N, int32_t T, hipStream_t stream)
{
    const size_t entries = (size_t)N + 1;
    std::unique_ptr<int32_t[]> h(new (std::nothrow) int32_t[entries]);
    if (!h) return KDA_ERR_LAUNCH;
    if (hipMemcpyAsync(h.get(), cu, sizeof(int32_t) * entries, hipMemcpyDeviceToHost, stream) != hipSuccess ||
        hipStreamSynchronize(stream) != hipSuccess)
        return KDA_ERR_LAUNCH;
    if (h[0] != 0 || h[N] > T) return KDA_ERR_INVALID_ARG;
    for (int32_t n = 0; n < N; ++n)
        if (h[n + 1] < h[n]) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// ---------------------------------------------------------------- argument checks of the operators
inline bool dtype_ok(kda_dtype dtype) { return dtype == KDA_F32 || dtype == KDA_BF16; }
inline size_t elem_size(kda_dtype dtype) { return dtype == KDA_BF16 ? 2 : 4; }

// A token array: present (unless it has no elements) and aligned to its type.
inline bool array_ok(const void *p, int64_t elems, size_t size) { return (p || elems == 0) && aligned(p, size); }

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
inline bool keep_apart(std::initializer_list<Out> outs, std::initializer_list<In> ins)
{
    for (const Out *o = outs.begin(); o != outs.end(); ++o) {
        for (const Out *other = outs.begin(); other != o; ++other)
            if (meet(*o, *other)) return false;
        for (const In *i = ins.begin(); i != ins.end(); ++i)
            if (meet(*o, *i) && !(o->may >> (i - ins.begin()) & 1 && o->p == i->p)) return false;
    }
    return true;
}

inline kda_status from_hip(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH; }

inline hipStream_t hip_stream(kda_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

// What the packed calls share: sizes, type, cu_seqlens.  The kernels look a
// tile beyond a token, and a wave beyond a sequence, in int32.
inline bool packed_ok(const int32_t *cu, int32_t N, int32_t T, int32_t D, kda_dtype dtype)
{
    return dtype_ok(dtype) && N >= 0 && N <= INT32_MAX - 65536 && T >= 0 && T <= INT32_MAX - 65536 && D > 0 && cu &&
           aligned(cu, 4);
}

inline bool workspace_ok(const void *ws, size_t bytes, size_t need, size_t align)
{
    return need == 0 || (ws && aligned(ws, align) && bytes >= need);
}

inline size_t cu_bytes(int32_t N) { return ((size_t)N + 1) * sizeof(int32_t); }

inline kda_status check_cu(const int32_t *cu, int32_t N, int32_t T, kda_stream_t stream)
{
    return validate_enabled() ? validate_cu(cu, N, T, hip_stream(stream)) : KDA_OK;
}

// Rows of an array in bytes: `rows` of `width`, `pitch` apart.
struct Rows {
    const void *p;
    int64_t rows, width, pitch;
};
inline Rows dense(const void *p, size_t n) { return {p, n ? 1 : 0, (int64_t)n, (int64_t)n}; }

// Whether two such arrays share a byte.  Of the same pitch, rows may lie between each
// other's (columns of one matrix); of different ones, the whole ranges count.
inline bool rows_meet(const Rows &a, const Rows &b)
{
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
    const auto span = [](const Rows &r) { return In{r.p, (size_t)((r.rows - 1) * r.pitch + r.width)}; };
    if (!meet(span(a), span(b))) return false;
    if (a.pitch != b.pitch || (a.rows == 1 && b.rows == 1)) return true;
    const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % a.pitch;
    const int64_t from = off < 0 ? off + a.pitch : off;   // where b's rows begin, from the beginning of one of a's
    return from < a.width || from + b.width > a.pitch;
}

// KDA_VALIDATE=1: the slots that a call writes, on the host: none in [0, num_slots) twice.
inline kda_status check_slots(const int32_t *slots, int32_t n, int32_t num_slots, kda_stream_t stream)
{
    if (!validate_enabled() || n == 0) return KDA_OK;
    std::unique_ptr<int32_t[]> h(new (std::nothrow) int32_t[n]);
    if (!h) return KDA_ERR_LAUNCH;
    if (hipMemcpyAsync(h.get(), slots, sizeof(int32_t) * n, hipMemcpyDeviceToHost, hip_stream(stream)) != hipSuccess ||
        hipStreamSynchronize(hip_stream(stream)) != hipSuccess)
        return KDA_ERR_LAUNCH;
    std::sort(h.get(), h.get() + n);
    for (int32_t i = 1; i < n; ++i)
        if (h[i] == h[i - 1] && h[i] >= 0 && h[i] < num_slots) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace kda_host

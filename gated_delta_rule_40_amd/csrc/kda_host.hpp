// kda_host.hpp -- host-side helpers shared by the C ABI's entry points:
// pointer alignment and the opt-in check of cu_seqlens.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <cstring>
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

}  // namespace kda_host

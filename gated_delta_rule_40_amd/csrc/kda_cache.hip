// kda_cache.hip -- entries of a cache of states in 8 or 4 bits, written from and
// read into rows of values.
//
// A thread moves pieces of 16 bytes of a row (four fp32 or eight bf16 values); the
// eight or four lanes that hold a block find its largest magnitude among them.
// What bounds both directions is HBM: 5 bytes a value (fp32, 8 bits), and one
// rounding of each.
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_mx.hpp"

namespace kda {

constexpr int CACHE_THREADS = 256;
constexpr int CACHE_PIECES = 4;   // of a thread

// The pieces of an entry, counted in whole blocks: the last ones may be parts or empty.
template <int VW> inline int64_t entry_pieces(int64_t elems) { return (elems + MXB - 1) / MXB * (MXB / VW); }

// Piece number `offset` after the first one of a workgroup, whose entry and
// place are known: a division of 32 bits.
struct Place {
    int64_t entry;
    uint32_t piece;
};
__device__ __forceinline__ Place place_of(int64_t entry0, uint32_t piece0, uint32_t offset, uint32_t per_entry)
{
    const uint32_t p = piece0 + offset;
    return {entry0 + p / per_entry, p % per_entry};
}

template <typename T, typename F>
__global__ __launch_bounds__(CACHE_THREADS) void kda_cache_store_kernel(const T *src, const int32_t *slots, int64_t entries,
                                                                        int32_t elems, uint32_t per_entry, int64_t entry_bytes,
                                                                        int32_t num_slots, uint8_t *cache, uint8_t *scales)
{
    constexpr int VW = 16 / sizeof(T), LANES = MXB / VW, BYTES = VW * F::BITS / 8;
    typedef T raw __attribute__((ext_vector_type(VW)));
    typedef raw mem __attribute__((aligned(sizeof(T))));
    const int64_t first = (int64_t)blockIdx.x * (CACHE_THREADS * CACHE_PIECES);
    const int64_t entry0 = first / per_entry;
    const uint32_t piece0 = (uint32_t)(first % per_entry);
    raw x[CACHE_PIECES];
    Place at[CACHE_PIECES];
    int count[CACHE_PIECES];
#pragma unroll
    for (int u = 0; u < CACHE_PIECES; ++u) {
        at[u] = place_of(entry0, piece0, threadIdx.x + u * CACHE_THREADS, per_entry);
        const int64_t begin = (int64_t)at[u].piece * VW;
        count[u] = at[u].entry < entries ? (int)max(min((int64_t)VW, elems - begin), (int64_t)0) : 0;
        x[u] = raw{};
        const T *p = src + at[u].entry * elems + begin;
        if (count[u] == VW) {
            x[u] = __builtin_nontemporal_load(reinterpret_cast<const mem *>(p));
        } else {
#pragma unroll
            for (int j = 0; j < VW; ++j)
                if (j < count[u]) x[u][j] = p[j];
        }
    }
#pragma unroll
    for (int u = 0; u < CACHE_PIECES; ++u) {
        float v[8] = {};
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            v[j] = to_f(x[u][j]);
            top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
        }
        top = max(top, dpp<DPP_XOR1>(top));
        top = max(top, dpp<DPP_XOR2>(top));
        if (LANES == 8) top = max(top, dpp<DPP_HALF_MIRROR>(top));
        const int sc = mx_scale_of<F>(top);
        const float up = mx_up(sc);
        uint32_t w[2];
        if (F::BITS == 4) {
            w[0] = F::encode(v, up);
        } else {
#pragma unroll
            for (int j = 0; j < VW / 4; ++j) w[j] = F::encode(v + 4 * j, up);
        }
        if (sc == 255) w[0] = w[1] = 0;
        if (count[u] == 0) continue;
        const int32_t slot = slots[at[u].entry];
        if (slot < 0 || slot >= num_slots) continue;
        if (at[u].piece % LANES == 0) scales[(int64_t)slot * (per_entry / LANES) + at[u].piece / LANES] = (uint8_t)sc;
        uint8_t *p = cache + slot * entry_bytes + (int64_t)at[u].piece * BYTES;
        if (count[u] == VW) {
            if (BYTES == 8) {
                typedef uint32_t two __attribute__((ext_vector_type(2)));
                typedef two two_mem __attribute__((aligned(1)));
                *reinterpret_cast<two_mem *>(p) = two{w[0], w[1]};
            } else if (BYTES == 4) {
                typedef uint32_t word_mem __attribute__((aligned(1)));
                *reinterpret_cast<word_mem *>(p) = w[0];
            } else {
                typedef uint16_t half_mem __attribute__((aligned(1)));
                *reinterpret_cast<half_mem *>(p) = (uint16_t)w[0];
            }
        } else {   // (values beyond the entry are zeros, and so is the half byte behind an odd one)
            const int n = (count[u] * F::BITS + 7) / 8;
#pragma unroll
            for (int j = 0; j < BYTES; ++j)
                if (j < n) p[j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
        }
    }
}

template <typename T, typename F>
__global__ __launch_bounds__(CACHE_THREADS) void kda_cache_load_kernel(const uint8_t *cache, const uint8_t *scales,
                                                                       const int32_t *slots, int64_t entries, int32_t elems,
                                                                       uint32_t per_entry, int64_t entry_bytes,
                                                                       int32_t num_slots, T *dst)
{
    constexpr int VW = 16 / sizeof(T), LANES = MXB / VW, BYTES = VW * F::BITS / 8;
    typedef T raw __attribute__((ext_vector_type(VW)));
    typedef raw mem __attribute__((aligned(sizeof(T))));
    const int64_t first = (int64_t)blockIdx.x * (CACHE_THREADS * CACHE_PIECES);
    const int64_t entry0 = first / per_entry;
    const uint32_t piece0 = (uint32_t)(first % per_entry);
    uint32_t w[CACHE_PIECES][2];
    int sc[CACHE_PIECES], count[CACHE_PIECES];
    Place at[CACHE_PIECES];
#pragma unroll
    for (int u = 0; u < CACHE_PIECES; ++u) {
        at[u] = place_of(entry0, piece0, threadIdx.x + u * CACHE_THREADS, per_entry);
        const int64_t begin = (int64_t)at[u].piece * VW;
        count[u] = at[u].entry < entries ? (int)max(min((int64_t)VW, elems - begin), (int64_t)0) : 0;
        w[u][0] = w[u][1] = 0;
        sc[u] = 127;
        const int32_t slot = count[u] ? slots[at[u].entry] : -1;
        if (slot < 0 || slot >= num_slots) continue;
        sc[u] = scales[(int64_t)slot * (per_entry / LANES) + at[u].piece / LANES];
        const uint8_t *p = cache + slot * entry_bytes + (int64_t)at[u].piece * BYTES;
        if (count[u] == VW) {
            if (BYTES == 8) {
                typedef uint32_t two __attribute__((ext_vector_type(2)));
                typedef two two_mem __attribute__((aligned(1)));
                const two q = *reinterpret_cast<const two_mem *>(p);
                w[u][0] = q[0], w[u][1] = q[1];
            } else if (BYTES == 4) {
                typedef uint32_t word_mem __attribute__((aligned(1)));
                w[u][0] = *reinterpret_cast<const word_mem *>(p);
            } else {
                typedef uint16_t half_mem __attribute__((aligned(1)));
                w[u][0] = *reinterpret_cast<const half_mem *>(p);
            }
        } else {
            const int n = (count[u] * F::BITS + 7) / 8;
#pragma unroll
            for (int j = 0; j < BYTES; ++j)
                if (j < n) w[u][j / 4] |= (uint32_t)p[j] << (8 * (j % 4));
        }
    }
#pragma unroll
    for (int u = 0; u < CACHE_PIECES; ++u) {
        float v[8];
        if (F::BITS == 4) {
            F::decode(w[u][0], v);
        } else {
#pragma unroll
            for (int j = 0; j < VW / 4; ++j) F::decode(w[u][j], v + 4 * j);
        }
        const float down = mx_down<F>(sc[u]);
        raw x;
#pragma unroll
        for (int j = 0; j < VW; ++j) x[j] = from_f<T>(v[j] * down);
        T *p = dst + at[u].entry * elems + (int64_t)at[u].piece * VW;
        if (count[u] == VW) {
            __builtin_nontemporal_store(x, reinterpret_cast<mem *>(p));
        } else {
#pragma unroll
            for (int j = 0; j < VW; ++j)
                if (j < count[u]) p[j] = x[j];
        }
    }
}

template <typename T> int64_t cache_groups(int32_t entries, int32_t elems)
{
    const int64_t pieces = entry_pieces<16 / (int)sizeof(T)>(elems) * entries, per = CACHE_THREADS * CACHE_PIECES;
    return (pieces + per - 1) / per;
}

}  // namespace kda

using namespace kda;

bool kda_cache_fits(bool bf16, int32_t entries, int32_t elems)
{
    return kda_grid_ok(bf16 ? cache_groups<bf16_t>(entries, elems) : cache_groups<float>(entries, elems), CACHE_THREADS);
}

template <typename T>
static hipError_t cache_store(const void *src, const int32_t *slots, int32_t entries, int32_t elems, int format,
                              int64_t entry_bytes, int32_t num_slots, uint8_t *cache, uint8_t *scales, hipStream_t s)
{
    return with_format(format, [&](auto f) {
        hipLaunchKernelGGL((kda_cache_store_kernel<T, decltype(f)>), dim3((unsigned)cache_groups<T>(entries, elems)),
                           dim3(CACHE_THREADS), 0, s, (const T *)src, slots, (int64_t)entries, elems,
                           (uint32_t)entry_pieces<16 / sizeof(T)>(elems), entry_bytes, num_slots, cache, scales);
        return hipGetLastError();
    });
}

hipError_t kda_launch_cache_store(bool bf16, const void *src, const int32_t *slots, int32_t entries, int32_t elems,
                                  int format, int64_t entry_bytes, int32_t num_slots, uint8_t *cache, uint8_t *scales,
                                  hipStream_t s)
{
    return bf16 ? cache_store<bf16_t>(src, slots, entries, elems, format, entry_bytes, num_slots, cache, scales, s)
                : cache_store<float>(src, slots, entries, elems, format, entry_bytes, num_slots, cache, scales, s);
}

template <typename T>
static hipError_t cache_load(const uint8_t *cache, const uint8_t *scales, const int32_t *slots, int32_t entries, int32_t elems,
                             int format, int64_t entry_bytes, int32_t num_slots, void *dst, hipStream_t s)
{
    return with_format(format, [&](auto f) {
        hipLaunchKernelGGL((kda_cache_load_kernel<T, decltype(f)>), dim3((unsigned)cache_groups<T>(entries, elems)),
                           dim3(CACHE_THREADS), 0, s, cache, scales, slots, (int64_t)entries, elems,
                           (uint32_t)entry_pieces<16 / sizeof(T)>(elems), entry_bytes, num_slots, (T *)dst);
        return hipGetLastError();
    });
}

hipError_t kda_launch_cache_load(bool bf16, const uint8_t *cache, const uint8_t *scales, const int32_t *slots,
                                 int32_t entries, int32_t elems, int format, int64_t entry_bytes, int32_t num_slots,
                                 void *dst, hipStream_t s)
{
    return bf16 ? cache_load<bf16_t>(cache, scales, slots, entries, elems, format, entry_bytes, num_slots, dst, s)
                : cache_load<float>(cache, scales, slots, entries, elems, format, entry_bytes, num_slots, dst, s);
}

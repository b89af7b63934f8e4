// kda_cache.hip -- entries of a cache of states in 8 or 4 bits, written from and
// read into rows of values.
//
// A thread moves pieces of 16 bytes of a row (four fp32 or eight bf16 values); the
// eight or four lanes that hold a block find its largest magnitude among them.  A
// value is rounded once.  HBM bounds both directions: one MI355X, 256 states of 32
// heads, fp32 and 8 bits (5.03 bytes a value), 114 us written and 113 read (5.9 TB/s);
// 777 entries of 6,003 bf16 in 4 bits 4.9 and 5.1 us.
#include "kda_device.hpp"
#include "kda_layer.hpp"
#include "kda_mx.hpp"

namespace kda {

constexpr int CACHE_THREADS = 256;
constexpr int CACHE_PIECES = 2;   // of a thread

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
            x[u] = *reinterpret_cast<const mem *>(p);
        } else {
#pragma unroll
            for (int j = 0; j < VW; ++j)
                if (j < count[u]) x[u][j] = p[j];
        }
    }
#pragma unroll
    for (int u = 0; u < CACHE_PIECES; ++u) {
        float v[8] = {};
        float largest = 0.f;
#pragma unroll
        for (int j = 0; j < VW; ++j) v[j] = to_f(x[u][j]), largest = mx_top(largest, v[j]);
        uint32_t top = __float_as_uint(largest) & 0x7fffffffu;   // (as bits a NaN is above all others)
        top = max(top, dpp<DPP_XOR1>(top));
        top = max(top, dpp<DPP_XOR2>(top));
        if (LANES == 8) top = max(top, dpp<DPP_HALF_MIRROR>(top));
        const int sc = mx_scale_of<F>(top);
        uint32_t w[2];
        if (F::BITS == 4) {
            w[0] = F::encode(v, sc);
        } else {
#pragma unroll
            for (int j = 0; j < VW / 4; ++j) w[j] = F::encode(v + 4 * j, sc);
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
            *reinterpret_cast<mem *>(p) = x;
        } else {
#pragma unroll
            for (int j = 0; j < VW; ++j)
                if (j < count[u]) p[j] = x[j];
        }
    }
}

// ---------------------------------------------------------------- entries of whole chunks
// A wave takes a chunk of 1,024 values of one entry, reads and writes 16 bytes a lane
// (of codes of 4 bits, 8), and hands the codes to the lanes that write or read them
// through LDS.  ONCE: past the caches, for calls too large to be found there again.
constexpr int CHUNK = 1024, CHUNK_WAVES = CACHE_THREADS / 64;

template <typename T, typename F> struct Chunk {
    static constexpr int VW = 16 / sizeof(T), PIECES = CHUNK / 64 / VW, LANES = MXB / VW;   // of a lane; lanes of a block
    static constexpr int PIECE_BYTES = VW * F::BITS / 8, LANE_BYTES = CHUNK / 64 * F::BITS / 8;
    typedef T raw __attribute__((ext_vector_type(VW)));
    typedef raw raw_mem __attribute__((aligned(sizeof(T))));
    typedef uint32_t words __attribute__((ext_vector_type(LANE_BYTES / 4)));
    typedef words words_mem __attribute__((aligned(1)));
    typedef uint32_t word_mem __attribute__((aligned(1)));
    // codes of the chunk in order, and its scales
    struct Shared {
        __attribute__((aligned(16))) uint8_t codes[64 * LANE_BYTES], scales[CHUNK / MXB];
    };
};

template <typename T, typename F, bool ONCE>
__global__ __launch_bounds__(CACHE_THREADS) void kda_cache_store_chunks_kernel(const T *src, const int32_t *slots, int64_t chunks,
                                                                               uint32_t per_entry, int32_t num_slots,
                                                                               uint8_t *cache, uint8_t *scales)
{
    typedef Chunk<T, F> C;
    __shared__ typename C::Shared shared[CHUNK_WAVES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t at = (int64_t)blockIdx.x * CHUNK_WAVES + wave;
    if (at >= chunks) return;
    typename C::raw x[C::PIECES];
#pragma unroll
    for (int k = 0; k < C::PIECES; ++k) {
        const auto *p = reinterpret_cast<const typename C::raw_mem *>(src + at * CHUNK + (k * 64 + lane) * C::VW);
        x[k] = ONCE ? __builtin_nontemporal_load(p) : *p;
    }
    const uint32_t entry = (uint32_t)at / per_entry;
    const int32_t slot = slots[entry];
    if (slot < 0 || slot >= num_slots) return;
    typename C::Shared &sh = shared[wave];
#pragma unroll
    for (int k = 0; k < C::PIECES; ++k) {
        float v[8] = {}, largest = 0.f;
#pragma unroll
        for (int j = 0; j < C::VW; ++j) v[j] = to_f(x[k][j]), largest = mx_top(largest, v[j]);
        uint32_t top = __float_as_uint(largest) & 0x7fffffffu;   // (as bits a NaN is above all others)
        top = max(top, dpp<DPP_XOR1>(top));
        top = max(top, dpp<DPP_XOR2>(top));
        if (C::LANES == 8) top = max(top, dpp<DPP_HALF_MIRROR>(top));
        const int sc = mx_scale_of<F>(top), finite = min(sc, 254);
        uint8_t *p = sh.codes + (k * 64 + lane) * C::PIECE_BYTES;
        if (__any(sc == 255)) {   // a block without a number: its codes are zeros
#pragma unroll
            for (int j = 0; j < C::VW; ++j) v[j] = sc == 255 ? 0.f : v[j];
        }
        if (C::PIECE_BYTES == 8) {
            reinterpret_cast<uint32_t *>(p)[0] = F::encode(v, finite), reinterpret_cast<uint32_t *>(p)[1] = F::encode(v + 4, finite);
        } else if (C::PIECE_BYTES == 4) {
            *reinterpret_cast<uint32_t *>(p) = F::encode(v, finite);
        } else {
            *reinterpret_cast<uint16_t *>(p) = (uint16_t)F::encode(v, finite);
        }
        if (lane % C::LANES == 0) sh.scales[k * (64 / C::LANES) + lane / C::LANES] = (uint8_t)sc;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int64_t to = (int64_t)slot * per_entry + (uint32_t)at % per_entry;   // chunks before
    const auto w = *reinterpret_cast<const typename C::words *>(sh.codes + lane * C::LANE_BYTES);
    auto *p = reinterpret_cast<typename C::words_mem *>(cache + to * (64 * C::LANE_BYTES) + lane * C::LANE_BYTES);
    if (ONCE) __builtin_nontemporal_store(w, p);
    else *p = w;
    if (lane < CHUNK / MXB / 4)
        *reinterpret_cast<typename C::word_mem *>(scales + to * (CHUNK / MXB) + 4 * lane) =
            *reinterpret_cast<const uint32_t *>(sh.scales + 4 * lane);
}

template <typename T, typename F, bool ONCE>
__global__ __launch_bounds__(CACHE_THREADS) void kda_cache_load_chunks_kernel(const uint8_t *cache, const uint8_t *scales,
                                                                              const int32_t *slots, int64_t chunks,
                                                                              uint32_t per_entry, int32_t num_slots, T *dst)
{
    typedef Chunk<T, F> C;
    __shared__ typename C::Shared shared[CHUNK_WAVES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t at = (int64_t)blockIdx.x * CHUNK_WAVES + wave;
    if (at >= chunks) return;
    const int32_t slot = slots[(uint32_t)at / per_entry];
    typename C::Shared &sh = shared[wave];
    typename C::words w{};
    uint32_t sc = 0x7f7f7f7f;
    if (slot >= 0 && slot < num_slots) {
        const int64_t from = (int64_t)slot * per_entry + (uint32_t)at % per_entry;   // chunks before
        const auto *p = reinterpret_cast<const typename C::words_mem *>(cache + from * (64 * C::LANE_BYTES) + lane * C::LANE_BYTES);
        w = ONCE ? __builtin_nontemporal_load(p) : *p;
        if (lane < CHUNK / MXB / 4) sc = *reinterpret_cast<const typename C::word_mem *>(scales + from * (CHUNK / MXB) + 4 * lane);
    }
    *reinterpret_cast<typename C::words *>(sh.codes + lane * C::LANE_BYTES) = w;
    if (lane < CHUNK / MXB / 4) *reinterpret_cast<uint32_t *>(sh.scales + 4 * lane) = sc;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int k = 0; k < C::PIECES; ++k) {
        const uint8_t *p = sh.codes + (k * 64 + lane) * C::PIECE_BYTES;
        const float down = mx_down<F>(sh.scales[k * (64 / C::LANES) + lane / C::LANES]);
        float v[8];
        if (C::PIECE_BYTES == 8) {
            F::decode(reinterpret_cast<const uint32_t *>(p)[0], v), F::decode(reinterpret_cast<const uint32_t *>(p)[1], v + 4);
        } else if (C::PIECE_BYTES == 4) {
            F::decode(*reinterpret_cast<const uint32_t *>(p), v);
        } else {
            F::decode(*reinterpret_cast<const uint16_t *>(p), v);
        }
        typename C::raw x;
#pragma unroll
        for (int j = 0; j < C::VW; ++j) x[j] = from_f<T>(v[j] * down);
        auto *to = reinterpret_cast<typename C::raw_mem *>(dst + at * CHUNK + (k * 64 + lane) * C::VW);
        if (ONCE) __builtin_nontemporal_store(x, to);
        else *to = x;
    }
}

// ---------------------------------------------------------------- host
// Entries of whole chunks go by chunks (256 states of 32 heads, fp32 and fp8: 114 us written,
// 113 read; 121 and 137 by pieces; 16 of 8 heads 3.2 and 3.7, 3.6 and 3.6 by pieces).
inline bool whole_chunks(int32_t entries, int32_t elems)
{
    return elems % CHUNK == 0 && (int64_t)entries * (elems / CHUNK) <= UINT32_MAX;
}

template <typename T> int64_t cache_groups(int32_t entries, int32_t elems)
{
    if (whole_chunks(entries, elems)) return ((int64_t)entries * (elems / CHUNK) + CHUNK_WAVES - 1) / CHUNK_WAVES;
    const int64_t pieces = entry_pieces<16 / (int)sizeof(T)>(elems) * entries, per = CACHE_THREADS * CACHE_PIECES;
    return (pieces + per - 1) / per;
}

// Whether a call's rows are too large to be found in the caches again (fp8 to fp32, past them
// and through them: 113 and 140 us for 537 MB, 4.1 and 3.6 for 8 MB).
template <typename T> bool past_caches(int32_t entries, int32_t elems) { return (int64_t)entries * elems * sizeof(T) > (64 << 20); }

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
        typedef decltype(f) F;
        const dim3 grid((unsigned)cache_groups<T>(entries, elems));
        if (whole_chunks(entries, elems)) {
            const auto kernel = past_caches<T>(entries, elems) ? kda_cache_store_chunks_kernel<T, F, true>
                                                               : kda_cache_store_chunks_kernel<T, F, false>;
            hipLaunchKernelGGL(kernel, grid, dim3(CACHE_THREADS), 0, s, (const T *)src, slots, (int64_t)entries * (elems / CHUNK),
                               (uint32_t)(elems / CHUNK), num_slots, cache, scales);
        } else {
            hipLaunchKernelGGL((kda_cache_store_kernel<T, F>), grid, dim3(CACHE_THREADS), 0, s, (const T *)src, slots,
                               (int64_t)entries, elems, (uint32_t)entry_pieces<16 / sizeof(T)>(elems), entry_bytes, num_slots,
                               cache, scales);
        }
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
        typedef decltype(f) F;
        const dim3 grid((unsigned)cache_groups<T>(entries, elems));
        if (whole_chunks(entries, elems)) {
            const auto kernel = past_caches<T>(entries, elems) ? kda_cache_load_chunks_kernel<T, F, true>
                                                               : kda_cache_load_chunks_kernel<T, F, false>;
            hipLaunchKernelGGL(kernel, grid, dim3(CACHE_THREADS), 0, s, cache, scales, slots, (int64_t)entries * (elems / CHUNK),
                               (uint32_t)(elems / CHUNK), num_slots, (T *)dst);
        } else {
            hipLaunchKernelGGL((kda_cache_load_kernel<T, F>), grid, dim3(CACHE_THREADS), 0, s, cache, scales, slots,
                               (int64_t)entries, elems, (uint32_t)entry_pieces<16 / sizeof(T)>(elems), entry_bytes, num_slots,
                               (T *)dst);
        }
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

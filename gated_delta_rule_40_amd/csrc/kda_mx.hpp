// kda_mx.hpp -- the formats of a cache of states: codes of 8 or 4 bits in blocks
// of 32 values that share a power-of-two scale (OCP microscaling formats).
//
// A format turns codes into the numbers they stand for and back.  raw(code) =
// number * 2^SHIFT is what its conversions give and take, so a value is
// raw * 2^(scale - 127 - SHIFT).  Scaling by a power of two is exact, and the
// conversions round to nearest, ties to even: a code is rounded once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int MXB = 32;   // values of a block

// A lane's value from another lane, without the LDS unit.
template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int CTRL> __device__ __forceinline__ float dpp(float x) { return __uint_as_float(dpp<CTRL>(__float_as_uint(x))); }
constexpr int DPP_XOR1 = 0xb1;          // quad_perm [1,0,3,2]
constexpr int DPP_XOR2 = 0x4e;          // quad_perm [2,3,0,1]
constexpr int DPP_HALF_MIRROR = 0x141;  // i -> 7 - i in groups of eight
constexpr int DPP_ROR8 = 0x128;         // i -> i ^ 8 in rows of 16

struct Fp8 {   // e4m3
    static constexpr int BITS = 8, SHIFT = 0, PLACES = 9;      // largest number 0.875 * 2^9
    static constexpr float TOP = 0.875f;
    // the raw numbers of a word's codes
    static __device__ __forceinline__ void decode(uint32_t w, float *v) {
        typedef float pair __attribute__((ext_vector_type(2)));
        const pair lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
    }
    // the codes of four values times `up` (2^(127 - scale))
    static __device__ __forceinline__ uint32_t encode(const float *v, float up) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * up, v[1] * up, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * up, v[3] * up, lo, true);
    }
};

struct Int8 {
    static constexpr int BITS = 8, SHIFT = 6, PLACES = 1;      // largest number 127/64 = 0.9921875 * 2^1
    static constexpr float TOP = 0.9921875f;
    static __device__ __forceinline__ void decode(uint32_t w, float *v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(w >> (8 * j));
    }
    static __device__ __forceinline__ uint32_t encode(const float *v, float up) {
        // v up is exact; times 64 plus 1.5 * 2^23 leaves the nearest integer in the low
        // bits, in one rounding.  Magnitudes above 127/64 (of blocks at the largest
        // scale alone) become that.
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            b[j] = __float_as_uint(__builtin_fmaf(__builtin_amdgcn_fmed3f(v[j] * up, -1.984375f, 1.984375f), 64.f, 12582912.f));
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0c);
        return lo | hi;
    }
};

struct Fp4 {   // e2m1
    static constexpr int BITS = 4, SHIFT = 0, PLACES = 3;      // largest number 6 = 0.75 * 2^3
    static constexpr float TOP = 0.75f;
    static __device__ __forceinline__ void decode(uint32_t w, float *v) {
        typedef float pair __attribute__((ext_vector_type(2)));
        const pair a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1),
                   c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3);
        v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
    }
    static __device__ __forceinline__ uint32_t encode(const float *v, float up) {
        uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, v[0] * up, v[1] * up, 1.f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * up, v[3] * up, 1.f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * up, v[5] * up, 1.f, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * up, v[7] * up, 1.f, 3);
    }
};

// The e8m0 byte of a block whose largest magnitude has these bits.
template <typename F> __device__ __forceinline__ int mx_scale_of(uint32_t amax_bits)
{
    if (amax_bits == 0) return 127;
    if (amax_bits >= 0x7f800000u) return 255;
    int e;
    const float m = frexpf(__uint_as_float(amax_bits), &e);   // amax = m 2^e, m in [1/2, 1)
    return min(max(e - F::PLACES + (m > F::TOP ? 1 : 0), -127), 127) + 127;
}
// 2^(127 - scale): values to numbers
__device__ __forceinline__ float mx_up(int scale) { return ldexpf(1.f, 127 - scale); }
// 2^(scale - 127 - SHIFT): raw numbers to values; NaN for the scale that is none
template <typename F> __device__ __forceinline__ float mx_down(int scale)
{
    return scale == 255 ? __builtin_nanf("") : ldexpf(1.f, scale - 127 - F::SHIFT);
}

// calls f with the format as a value of its type
template <typename Fn> auto with_format(int format, Fn f)
{
    return format == 0 ? f(Fp8()) : format == 1 ? f(Int8()) : f(Fp4());
}

}  // namespace kda

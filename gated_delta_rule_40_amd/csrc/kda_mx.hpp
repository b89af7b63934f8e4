// kda_mx.hpp -- the formats of a cache of states: codes of 8 or 4 bits in blocks
// of 32 values that share a power-of-two scale (OCP microscaling formats).
//
// A format turns codes into the numbers they stand for and back.  raw(code) =
// number * 2^SHIFT is what its conversions give and take, so a value is
// raw * 2^(scale - 127 - SHIFT).  Scaling by a power of two is exact, and the
// conversions round to nearest, ties to even: a code is rounded once.
#pragma once

#include "kda_lanes.hpp"

namespace kda {

constexpr int MXB = 32;   // values of a block

// decode: the raw numbers of a word's codes.  encode: the codes of a word's values
// in a block with this scale byte (0 to 254).  The scaled conversions take a scale
// as the exponent of a float, byte 0 (2^-127) too.
struct Fp8 {   // e4m3
    static constexpr int BITS = 8, SHIFT = 0, PLACES = 9;      // largest number 0.875 * 2^9
    static constexpr float TOP = 0.875f;
    static __device__ __forceinline__ void decode(uint32_t w, float *v) {
        typedef float pair __attribute__((ext_vector_type(2)));
        const pair lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
    }
    static __device__ __forceinline__ uint32_t encode(const float *v, int scale) {
        typedef short two __attribute__((ext_vector_type(2)));
        const float s = __uint_as_float((uint32_t)scale << 23);
        two w;
        asm("" : "=v"(w));   // (both halves are written below)
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[0], v[1], s, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[2], v[3], s, true);
        return __builtin_bit_cast(uint32_t, w);
    }
};

struct Int8 {
    static constexpr int BITS = 8, SHIFT = 6, PLACES = 1;      // largest number 127/64 = 0.9921875 * 2^1
    static constexpr float TOP = 0.9921875f;
    static __device__ __forceinline__ void decode(uint32_t w, float *v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (float)(int8_t)(w >> (8 * j));
    }
    static __device__ __forceinline__ uint32_t encode(const float *v, int scale) {
        // 64 numbers plus 1.5 * 2^23: the nearest integer is in the low bits, in one rounding
        constexpr float magic = 12582912.f;
        float r[4];
        if (scale >= 6 && scale < 254) {
            const float up = __uint_as_float((uint32_t)(260 - scale) << 23);   // 64 * 2^(127 - scale)
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = __builtin_fmaf(v[j], up, magic);
        } else {   // that is no float, or values may be above 127/64 (and become that)
            const float up = ldexpf(1.f, 127 - scale);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[j] = __builtin_fmaf(__builtin_amdgcn_fmed3f(v[j] * up, -1.984375f, 1.984375f), 64.f, magic);
        }
        const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(r[1]), __float_as_uint(r[0]), 0x0c0c0400);
        const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(r[3]), __float_as_uint(r[2]), 0x04000c0c);
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
    static __device__ __forceinline__ uint32_t encode(const float *v, int scale) {
        const float s = __uint_as_float((uint32_t)scale << 23);
        uint32_t w;
        asm("" : "=v"(w));   // (all four bytes are written below)
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
    }
};

// The largest magnitude, a NaN if there is one.
__device__ __forceinline__ float mx_top(float a, float b) { return __builtin_elementwise_maximum(a, __builtin_fabsf(b)); }

// The e8m0 byte of a block whose largest magnitude has these bits: the exponent, one
// more where the mantissa is above the largest number's (bits FRACTION), less PLACES.
template <typename F> __device__ __forceinline__ int mx_scale_of(uint32_t amax_bits)
{
    constexpr uint32_t FRACTION = (uint32_t)((F::TOP * 2.f - 1.f) * 8388608.f);
    int e = (int)((amax_bits + (0x7fffffu - FRACTION)) >> 23) + (1 - F::PLACES);
    if (F::PLACES == 1) {   // the others never reach the ends
        if (amax_bits <= 0x7f0000u) e = 0;   // (below 2^-126 the bits are no exponent and mantissa)
        e = min(e, 254);
    }
    e = max(e, 0);
    e = amax_bits == 0 ? 127 : e;
    return amax_bits >= 0x7f800000u ? 255 : e;
}
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

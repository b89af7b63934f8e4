// kda_lanes.hpp -- values from other lanes of a wave, without the LDS unit.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int CTRL> __device__ __forceinline__ float dpp(float x) { return __uint_as_float(dpp<CTRL>(__float_as_uint(x))); }
constexpr int DPP_XOR1 = 0xb1;          // quad_perm [1,0,3,2]
constexpr int DPP_XOR2 = 0x4e;          // quad_perm [2,3,0,1]
constexpr int DPP_HALF_MIRROR = 0x141;  // i -> 7 - i in groups of eight
constexpr int DPP_REVERSE4 = 0x1b;      // quad_perm [3,2,1,0]
constexpr int DPP_MIRROR = 0x140;       // i -> 15 - i in rows of 16
constexpr int DPP_ROR8 = 0x128;         // i -> i ^ 8 in rows of 16

// x of lane l plus x of lane l ^ 16, and l ^ 32
__device__ __forceinline__ float add_xor16(float x)
{
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float add_xor32(float x)
{
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

}  // namespace kda

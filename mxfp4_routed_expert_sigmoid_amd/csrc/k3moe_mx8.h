// MXFP8 tokens (e4m3 values, one E8M0 byte per 32 of a row), as the norm and
// the dense products write them: per group the smallest power of two 2^s,
// s >= -127, with max|v| <= 448 * 2^s over the group's finite values, byte
// s + 127, and e4m3_RNE(v / 2^s). No value is clipped (448 is the largest
// e4m3), so each is off by at most half a step; dividing by 2^s is exact
// down to values that round to zero. A value that is not finite is stored as
// NaN and takes no part in the maximum.
#pragma once

#include "k3moe_device.h"

namespace k3moe {

// s of a group whose largest finite magnitude is m (m >= 0, finite).
__device__ __forceinline__ int mx8_exp(float m)
{
    const uint32_t u = __float_as_uint(m);
    // m = 1.f * 2^(e - 127) (a subnormal m lies far below 448 * 2^-127):
    // m <= 1.75 * 2^(s + 8) with the smallest s
    const int e = (int)(u >> 23);
    const int s = e - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return s < -127 ? -127 : s;
}

// 2^-s as a factor: s in [-127, 120], so it is a normal fp32 number.
__device__ __forceinline__ float mx8_inv(int s) { return __uint_as_float((uint32_t)(127 - s) << 23); }

__device__ __forceinline__ float mx8_mag(float v)
{
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.0f;  // inf and NaN: 0
}

// The e4m3 code of v / 2^s (inv = 2^-s), to nearest even.
__device__ __forceinline__ uint32_t mx8_code(float v, float inv)
{
    const uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v * inv, 0.0f, 0, false) & 0xffu;
    return fabsf(v) < INFINITY ? c : 0x7fu;
}

// Maximum over each aligned run of 32 lanes.
__device__ __forceinline__ float half_wave_max(float m)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    return m;
}

}  // namespace k3moe

// The 8-bit form of a block of values, shared by the kernels that write or read
// it (gfx950 only): scale = max|x| / 127 in fp32, code = x / scale to nearest.
#pragma once
#include "kda_device.h"

namespace kda {

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kAct8Tiny = 1.17549435e-38f;    // 2^-126: 1 / scale stays finite
constexpr float kAct8Huge = 2.67938851e36f;     // largest scale with 127 * scale finite

// The largest magnitude is taken over the bit patterns without their sign: as
// whole numbers they order finite values, then infinity, then NaN, so a value
// that is not finite is never lost.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

__device__ __forceinline__ float act8_scale(uint32_t amax_bits) {
    if (amax_bits >= kInfBits) return __builtin_nanf("");
    return fminf(fmaxf(__builtin_bit_cast(float, amax_bits) / 127.f, kAct8Tiny), kAct8Huge);
}

// x / s rounded to nearest, ties of the exact quotient to even.  The product
// with the reciprocal can land on the wrong side of the middle of two codes; the
// remainder x - q s is exact in fp32 (a multiple of ulp(s) or of ulp(s) / 2, at
// most about s), so comparing twice the remainder with s puts q right.
__device__ __forceinline__ int act8_code(float x, float s, float inv) {
    float q = rintf(x * inv);
    const float r2 = 2.f * fmaf(-q, s, x);
    const bool odd = ((int)q & 1) != 0;
    if (r2 > s || (r2 == s && odd)) q += 1.f;
    else if (r2 < -s || (r2 == -s && odd)) q -= 1.f;
    return (int)q;
}

__device__ __forceinline__ float act8_value(int8_t c, float s) { return (float)c * s; }

}  // namespace kda

// The 8-bit form of a block of values, shared by the kernels that write or read
// it (gfx950 only): scale = max|x| (1 / 127) in fp32, code = x / scale to nearest.
#pragma once
#include <type_traits>

#include "kda_device.h"

namespace kda {

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kAct8Tiny = 1.17549435e-38f;    // 2^-126: 1 / scale stays finite
// 1 / 127 to nearest is 127's exact inverse to 4e-9: 127 scales are max|x| to half a
// step of fp32, and finite for every finite max|x|.
constexpr float kAct8Step = 1.f / 127.f;

// The largest magnitude is taken over the bit patterns without their sign: as
// whole numbers they order finite values, then infinity, then NaN, so a value
// that is not finite is never lost.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

__device__ __forceinline__ float act8_scale(uint32_t amax_bits) {
    if (amax_bits >= kInfBits) return __builtin_nanf("");
    return fmaxf(__builtin_bit_cast(float, amax_bits) * kAct8Step, kAct8Tiny);
}

// x / s rounded to nearest, ties of the exact quotient to even.  The product with
// the reciprocal can land on the wrong side of the middle of two codes (half the
// block's largest magnitude is such a middle); the remainder x - q s is exact in
// fp32 (a multiple of ulp(s) or of ulp(s) / 2, at most about s), so comparing it
// with s / 2 puts q right.
__device__ __forceinline__ int act8_code(float x, float s, float inv) {
    const float q = rintf(x * inv), r = fmaf(-q, s, x), half = 0.5f * s;
    const int c = (int)q;
    const bool next = fabsf(r) > half || (fabsf(r) == half && (c & 1));
    return next ? c + (r > 0.f ? 1 : -1) : c;
}

__device__ __forceinline__ float act8_value(int8_t c, float s) { return (float)c * s; }

// Eight consecutive values at any element's address, as fp32.
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
template <typename X> struct Eight;
template <> struct Eight<bf16_t> {
    bf16x8_t v;
    __device__ __forceinline__ void load(const bf16_t *p) {
        typedef bf16x8_t at __attribute__((aligned(2)));
        v = __builtin_nontemporal_load(reinterpret_cast<const at *>(p));
    }
    __device__ __forceinline__ void load_kept(const bf16_t *p) {
        typedef bf16x8_t at __attribute__((aligned(2)));
        v = *reinterpret_cast<const at *>(p);
    }
    __device__ __forceinline__ float get(int e) const { return (float)v[e]; }
    __device__ __forceinline__ void set(int e, float x) { v[e] = (bf16_t)x; }
    __device__ __forceinline__ void store(bf16_t *p) const {
        typedef bf16x8_t at __attribute__((aligned(2)));
        __builtin_nontemporal_store(v, reinterpret_cast<at *>(p));
    }
};
template <> struct Eight<float> {
    f32x4_t v[2];
    __device__ __forceinline__ void load(const float *p) {
        typedef f32x4_t at __attribute__((aligned(4)));
        v[0] = __builtin_nontemporal_load(reinterpret_cast<const at *>(p));
        v[1] = __builtin_nontemporal_load(reinterpret_cast<const at *>(p) + 1);
    }
    __device__ __forceinline__ void load_kept(const float *p) {
        typedef f32x4_t at __attribute__((aligned(4)));
        v[0] = reinterpret_cast<const at *>(p)[0];
        v[1] = reinterpret_cast<const at *>(p)[1];
    }
    __device__ __forceinline__ float get(int e) const { return v[e / 4][e % 4]; }
    __device__ __forceinline__ void set(int e, float x) { v[e / 4][e % 4] = x; }
    __device__ __forceinline__ void store(float *p) const {
        typedef f32x4_t at __attribute__((aligned(4)));
        __builtin_nontemporal_store(v[0], reinterpret_cast<at *>(p));
        __builtin_nontemporal_store(v[1], reinterpret_cast<at *>(p) + 1);
    }
};
// Eight codes: kept as loaded until they are used.
struct Codes8 {
    u32x2_t w;
    __device__ __forceinline__ void load(const int8_t *p) {
        typedef u32x2_t at __attribute__((aligned(1)));
        w = __builtin_nontemporal_load(reinterpret_cast<const at *>(p));
    }
    __device__ __forceinline__ int8_t get(int e) const { return (int8_t)(w[e / 4] >> (8 * (e % 4))); }
    __device__ __forceinline__ void store(int8_t *p) const {
        typedef u32x2_t at __attribute__((aligned(1)));
        __builtin_nontemporal_store(w, reinterpret_cast<at *>(p));
    }
};

// The largest of x over 16 (or 8) neighbouring lanes, in each of them.
template <int LANES> __device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
    static_assert(LANES == 8 || LANES == 16, "lanes of a row of 16");
    const auto step = [&](auto ctrl) {
        x = max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, decltype(ctrl)::value, 0xf, 0xf, true));
    };
    step(std::integral_constant<int, 0xB1>());    // quad_perm [1,0,3,2]
    step(std::integral_constant<int, 0x4E>());    // quad_perm [2,3,0,1]
    step(std::integral_constant<int, 0x141>());   // row_half_mirror
    if constexpr (LANES == 16) step(std::integral_constant<int, 0x140>());   // row_mirror
    return x;
}

// The codes of eight values under a scale; a scale that is not finite gives zeros.
__device__ __forceinline__ Codes8 act8_codes(const float (&v)[8], float s) {
    const float inv = 1.f / s;
    const bool bad = !(s < __builtin_inff());
    Codes8 c;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= ((uint32_t)act8_code(v[4 * k + e], s, inv) & 0xffu) << (8 * e);
        c.w[k] = bad ? 0 : w;
    }
    return c;
}

}  // namespace kda

// ssd_code8.h -- values in 8 bits with one fp32 scale for a run of them: v / scale rounded to a code of int8 or e4m3
// (the state cache's groups; the norm's rows, whose quotients are of 64 bits).
#pragma once

#include "ssd_device.h"

namespace ssd {

constexpr float kMinScale = 0x1p-80f;  // below it the remainder of a quotient next to a border could leave the fp32 range

// v / s for a rounding to fewer bits: an fp32 quotient whose last bit is set when it is not exact, cut towards
// zero ("rounded to odd").  Rounding it again to 8 bits or fewer gives the exact quotient's nearest code; rounding a
// quotient that was itself rounded to nearest could fall on a border between two codes that the exact quotient
// only comes close to.  q is within a step of the exact quotient (one correction of v * inv, inv = 1 / s of the
// group), and the remainder v - q s, exact in one fma, says on which side.  (With a division a value instead of one
// a group the write took 20 us against 13 us at 16 x 655360 fp32 values.)
__device__ inline float quotient_to_odd(float v, float s, float inv) {
    const float q0 = v * inv;
    const float q = __builtin_fmaf(__builtin_fmaf(-q0, s, v), inv, q0);
    const float r = __builtin_fmaf(-q, s, v);
    uint32_t u = __builtin_bit_cast(uint32_t, q);
    const bool above = (r < 0.f) != (q < 0.f);  // |q| is above the exact quotient: step back
    // (a quotient too small for fp32 is 0 and has no step before it)
    u = (r != 0.f && q != 0.f) ? (above ? u - 1 : u) | 1u : u;
    return __builtin_bit_cast(float, u);
}

__device__ inline uint32_t code_int8(float q) {
    return (uint32_t)(int)rintf(fminf(fmaxf(q, -127.f), 127.f)) & 0xffu;
}

// e4m3 of a clamped quotient: the nearest multiple of the step at its magnitude, ties to even.
__device__ inline uint32_t code_e4m3(float q) {
    const uint32_t sign = __builtin_bit_cast(uint32_t, q) >> 31 << 7;
    const float m = fminf(fabsf(q), 448.f);
    int e = (int)(__builtin_bit_cast(uint32_t, m) >> 23) - 127;
    e = e < -6 ? -6 : e;
    // m / 2^(e-3) is below 16, so adding 1.5 * 2^23 rounds it to an integer, ties to even
    const float k = m * __builtin_bit_cast(float, (uint32_t)(127 + 3 - e) << 23) + 12582912.f;
    const int n = (int)(__builtin_bit_cast(uint32_t, k) & 0x3fffffu);  // 0 .. 16, in steps of 2^(e-3)
    // n = 8 + mantissa in the binade e (0 .. 7: the subnormal one); 16 carries into the next binade
    return sign | (uint32_t)((e + 6) * 8 + n);
}

__device__ inline float value_e4m3(uint32_t c) {
    const int e = (c >> 3) & 15, m = c & 7;
    if (e == 15 && m == 7) return __builtin_nanf("");
    const float v = e ? __builtin_bit_cast(float, (uint32_t)(e + 120) << 23 | (uint32_t)m << 20) : (float)m * 0x1p-9f;
    return c & 0x80u ? -v : v;
}

}  // namespace ssd

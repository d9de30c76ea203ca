// e4m3 numbers and their e8m0 scales in registers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace xs {

constexpr int LEAST_SCALE = 63;   // the smallest scale byte that is written: 2^-64

// A row's probabilities are taken relative to 2^-7 of the running maximum of probability times scale: as fp16 numbers
// they then reach from the type's upper end (2^15, the maximum having risen by 2^8 since) down to 2^-32 of the
// maximum; relative to the maximum itself they ended at 2^-25, and what many small ones add up to was lost.  (Two
// chunks of 2048 tokens over 16384 keys 786 us -> 789, few tokens the same.)
constexpr float HEADROOM = 7.0f;

// 2^(byte - 127), byte 1 .. 254
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// The same of any byte: 0 is 2^-127, a subnormal, 255 NaN.
__device__ __forceinline__ float any_scale_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fffffffu : byte << 23);
}

// 2^(127 - byte), byte 1 .. 254 (254: 2^-127, a subnormal)
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float(max((254u - byte) << 23, 0x00400000u)); }

// Scale byte of values up to `largest` (the bits of a non-negative float): the least s >= 63 with
// largest <= 448 * 2^(s - 127) = 1.75 * 2^(s - 119).  The sum carries into the exponent if the
// significand is above 1.75.
__device__ __forceinline__ int scale_byte(uint32_t largest) {
    const int s = static_cast<int>((largest + 0x1fffffu) >> 23) - 8;
    return s > LEAST_SCALE ? s : LEAST_SCALE;
}

// A row of Q as numbers: the exponent byte of the least scale whose 448-fold holds its largest magnitude, 2^-126 at least,
// and the inverse; NaN for an infinity (whose number would be 448 and its scores finite).
__device__ __forceinline__ int row_scale(float largest, float& inverse) {
    const int e = max(static_cast<int>((__float_as_uint(largest) + 0x1fffffu) >> 23) - 8, 1);
    inverse = largest <= 3.402823466e38f ? scale_value(254 - e) : __uint_as_float(0x7fffffffu);
    return e;
}

// Two e4m3 numbers (a byte each) as two fp16 ones: exact.
__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(r) : "r"(two));
    return r;
}

__device__ __forceinline__ uint32_t codes_to_f16x2_high(uint32_t four) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(r) : "r"(four));
    return r;
}

// Four values to the nearest e4m3 numbers (ties to even), the first in the lowest byte.
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\ncvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        "mov.b32 %0, {lo, hi};\n}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ float2 f16x2_values(uint32_t w) {
    float2 f;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.f32.f16 %0, lo;\ncvt.f32.f16 %1, hi;\n}" : "=f"(f.x), "=f"(f.y) : "r"(w));
    return f;
}

}  // namespace xs

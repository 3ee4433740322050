// mx_common.cuh -- microscaled (MX) blocks: 32 consecutive elements of a row share
// one E8M0 scale, the power of two 2^(code - 127).
//
// With m the block's largest magnitude, the scale is 2^(floor(log2 m) - emax), clamped
// to 2^-127 .. 2^127, where emax is the exponent of the element format's largest
// value (E2M1: 6 = 1.5 * 2^2; E4M3: 448 = 1.75 * 2^8).  Elements are value / scale
// rounded to the nearest format value, ties to even; magnitudes beyond the largest
// value saturate to it.  On fp32 bit patterns: floor(log2 m) + 127 is m's exponent
// field, so the scale code is that field minus emax (0 where it would be negative,
// subnormal m included), and the division by the scale is the exact product with
// 2^(127 - code).  A block that holds an infinity or a NaN has exponent field 255: its
// scale code is 255 (NaN), and every element reads as NaN.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {
namespace mx {

constexpr int kBlock = 32;      // elements per scale
constexpr int kEmaxE2M1 = 2;
constexpr int kEmaxE4M3 = 8;
constexpr uint32_t kNanScale = 255;

// E8M0 code of a block whose largest magnitude has the fp32 bits `max_bits` (sign bit clear).
__device__ __forceinline__ uint32_t scale_code(uint32_t max_bits, int emax)
{
    const int field = (int)(max_bits >> 23);
    return field == 255 ? kNanScale : (uint32_t)max(field - emax, 0);
}

// 2^(127 - code), the exact reciprocal of the scale (code <= 254 - emax).
__device__ __forceinline__ float inverse_scale(uint32_t code)
{
    return __uint_as_float((254u - code) << 23);
}

// Four fp32 values as E4M3 codes, v[0] in the lowest byte; round to nearest even,
// saturating at 448.
__device__ __forceinline__ uint32_t e4m3x4(float v0, float v1, float v2, float v3)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
    return r;
}

// Eight fp32 values as E2M1 codes, v[0] in the lowest nibble; round to nearest
// even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The largest magnitude's bits over the 4 consecutive lanes that hold one block.
// Magnitudes compare as integers, and every NaN is above every number.
__device__ __forceinline__ uint32_t quad_max(uint32_t bits)
{
    bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
    return max(bits, __shfl_xor_sync(0xffffffffu, bits, 2));
}

// The bits of the largest magnitude of 8 values, above every number's if one is a NaN.
__device__ __forceinline__ uint32_t max_bits(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// Quantises 8 consecutive values of a block spread over 4 consecutive lanes (all 32
// lanes take part); `m` is their max_bits.  `codes` gets 8 E4M3 bytes (E2M1: 8 nibbles in codes.x); returns
// the block's scale code.
template <bool E2M1>
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], uint32_t m, uint2& codes)
{
    m = quad_max(m);
    const uint32_t code = scale_code(m, E2M1 ? kEmaxE2M1 : kEmaxE4M3);
    if (code == kNanScale) {
        // E4M3 has a NaN code; E2M1 has none and leaves it to the scale
        codes = E2M1 ? make_uint2(0u, 0u) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        return code;
    }
    const float inv = inverse_scale(code);
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = v[i] * inv;
    if constexpr (E2M1) {
        codes = make_uint2(e2m1x8(u), 0u);
    } else {
        codes = make_uint2(e4m3x4(u[0], u[1], u[2], u[3]), e4m3x4(u[4], u[5], u[6], u[7]));
    }
    return code;
}

}  // namespace mx
}  // namespace moe

// Power-of-two block scales and the conversion to 8-bit floating point, shared
// by the casts and the product of few rows (the rule stands in fp8_cast.cu).
#pragma once

#include <cstdint>

namespace gns {

// Biased exponent of the scale of a block with this amax (finite, >= 0): with
// amax = 1.m 2^e, s = 2^(e - top) if 1.m <= 1.75 and twice that otherwise.
__device__ __forceinline__ uint32_t scale_exponent(float amax, int top) {
    const int b = static_cast<int>((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - top;
    return static_cast<uint32_t>(b < 1 ? 1 : b);
}
// 1 / 2^(biased - 127); biased <= 247, so the inverse is a normal number.
__device__ __forceinline__ float exp_inverse(uint32_t biased) { return __uint_as_float((254u - biased) << 23); }

// Four values as the bytes of a word, the first lowest.
template <bool E5M2>
__device__ __forceinline__ uint32_t cast_quad(float a, float b, float c, float d) {
    uint32_t r;
    if constexpr (E5M2)
        asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.0f;
}

// NaN for an infinity (the conversion saturates it), v otherwise.
__device__ __forceinline__ float no_infinity(float v) { return fabsf(v) == INFINITY ? __uint_as_float(0x7FC00000u) : v; }

}  // namespace gns

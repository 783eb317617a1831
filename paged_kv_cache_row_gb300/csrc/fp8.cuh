// fp8.cuh -- the 8-bit pool's formats: e4m3 elements and a power of two for
// each block of tokens and head (one byte e, for 2^(e - 127)).
//
// A power of two, because an element keeps its 4 significant bits whatever it
// is multiplied with: an element times its block's scale is exact in fp32 and
// bf16, a block's older rows change their scale without a rounding (but for
// elements that become subnormal), and no quotient is ever formed.
#pragma once
#include <cstdint>

#include "fp4.cuh"

namespace minisgl {
namespace fp8 {

constexpr int EXP_LOW = -120, EXP_HIGH = 119;  // exponents that a store gives
constexpr int EXP_BIAS = 127;

// The smallest e in range with a <= 448 * 2^e, for a >= 0 given by its fp32
// bits (448 = 1.75 * 2^8).
__device__ __forceinline__ int exponent_for(uint32_t bits) {
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, EXP_LOW), EXP_HIGH);
}

// 4 floats -> 4 e4m3 bytes, nearest (ties to even), saturating at 448; NaN -> 0x7f
__device__ __forceinline__ uint32_t f32_to_e4m3x4(float a, float b, float c, float d) {
    uint32_t w;
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
        " mov.b32 %0, {l, h};\n}\n"
        : "=r"(w)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}

// 4 e4m3 bytes -> 2 fp16 pairs (exact)
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

}  // namespace fp8
}  // namespace minisgl

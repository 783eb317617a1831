// fp4.cuh -- conversions between bf16 / fp16 and the 4-bit pool's formats:
// e2m1 elements (two to a byte, the first in the low half) and e4m3 scales.
// Each wrapper is one conversion instruction of sm_103a or a few of them.
//
// An element (at most 2 significant bits, 0.5 .. 6) times a scale (at most 4,
// 2^-9 .. 448) has at most 6 significant bits and lies between 2^-10 and
// 2688: it is exact in fp16, and times a power of two exact in bf16.
#pragma once
#include <cstdint>

namespace minisgl {

constexpr int FP4_BLOCK = 16;  // channels that share a scale

// 4 bytes of e2m1 pairs -> 4 fp16 pairs
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// 8 floats -> 4 bytes of e2m1 pairs, nearest (ties to even), saturating at 6
__device__ __forceinline__ uint32_t f32_to_e2m1x8(const float *x) {
    uint32_t w;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
        : "=r"(w)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return w;
}

// two e4m3 bytes (low 16 bits of x) -> fp16 pair
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
    uint32_t h;
    const uint16_t s = static_cast<uint16_t>(x);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(s));
    return h;
}

// float -> e4m3 byte, nearest (ties to even), saturating at 448; NaN -> 0x7f
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint16_t s;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(s) : "f"(0.f), "f"(x));
    return s & 0xffu;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

// a times one half of b, the low or the high (the multiplication can take either
// half twice, so that no permutation is needed first)
template <bool HIGH>
__device__ __forceinline__ uint32_t mul_f16x2_half(uint32_t a, uint32_t b) {
    uint32_t c;
    if constexpr (HIGH)
        asm("{\n .reg .b16 l, h;\n .reg .b32 s;\n mov.b32 {l, h}, %2;\n mov.b32 s, {h, h};\n"
            " mul.rn.f16x2 %0, %1, s;\n}\n" : "=r"(c) : "r"(a), "r"(b));
    else
        asm("{\n .reg .b16 l, h;\n .reg .b32 s;\n mov.b32 {l, h}, %2;\n mov.b32 s, {l, l};\n"
            " mul.rn.f16x2 %0, %1, s;\n}\n" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
    float2 f;
    asm("{\n .reg .f16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}\n"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

__device__ __forceinline__ uint32_t f32_to_f16x2(float lo, float hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace minisgl

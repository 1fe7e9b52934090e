// mx8.cuh -- microscaled 8-bit numbers: e4m3 codes, one power-of-two scale for 32 of
// them along a row.
//
//   scale 2^(s-127), the smallest with amax <= 448 2^(s-127)  (s >= 0; 255: Inf or NaN)
//   code = x 2^(127-s), rounded to the nearest e4m3, ties to the even code
//
// amax / scale lies in (224, 448], so that no code is clipped and each is within half an
// e4m3 step of its element (2^-4 of it, or 2^-10 of the scale for the smallest).  With
// the scale at the exponent of amax alone an eighth of all blocks would have their
// largest elements clipped, by up to an eighth.  All steps are exact but the rounding.
#pragma once
#include "common.cuh"

namespace moe {

// bytes of a row of scales: K / 32, in whole 16-byte pieces (512 elements each)
__host__ __device__ inline int64_t mx8_pitch(int64_t K) { return (K / 32 + 15) / 16 * 16; }

// scale byte of a block whose largest magnitude has these bits (Inf, NaN: 255).  The
// sum carries into the exponent where the mantissa is above 1.75 = 448 / 256.
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t amax_bits) {
    const uint32_t e = (amax_bits + 0x1fffffu) >> 23;
    return amax_bits >= 0x7f800000u ? 255u : (e > 8 ? e - 8 : 0u);
}
// 2^(127 - s): what a block's elements are multiplied by (0 for s = 255)
__device__ __forceinline__ float mx8_inv_scale(uint32_t s) { return __uint_as_float(s == 255 ? 0u : (254 - s) << 23); }
// 2^(s - 127), NaN for s = 255
__device__ __forceinline__ float mx8_scale_value(uint32_t s) {
    return __uint_as_float(s == 255 ? 0x7fc00000u : s == 0 ? 0x00400000u : s << 23);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// bits of the largest magnitude of N (even) values: NaN's where one is, which is above
// every number's; two values an instruction
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <int N>
__device__ __forceinline__ uint32_t amax_bits(const float* v) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; i += 2) m = max3_abs(m, v[i], v[i + 1]);
    return __float_as_uint(m);
}

// 4 scaled values -> 4 codes, the first in the low byte
__device__ __forceinline__ uint32_t mx8_pack4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\n"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        "mov.b32 %0, {lo, hi};\n}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
// N (a multiple of 4) values -> N / 4 words of codes.  A block of byte 255 holds Inf or
// NaN, and 0 times those is no number: its codes are set to 0.
template <int N>
__device__ __forceinline__ void mx8_codes(const float* v, uint32_t s, uint32_t* w) {
    const float m = mx8_inv_scale(s);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const uint32_t c = mx8_pack4(v[4 * i] * m, v[4 * i + 1] * m, v[4 * i + 2] * m, v[4 * i + 3] * m);
        w[i] = s == 255 ? 0u : c;
    }
}
// a word of 4 codes -> 4 values, without the scale (exact in fp16)
__device__ __forceinline__ void mx8_unpack4(uint32_t w, float* v) {
    uint32_t lo, hi;
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\n"
        "cvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}" : "=f"(v[0]), "=f"(v[1]) : "r"(lo));
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}" : "=f"(v[2]), "=f"(v[3]) : "r"(hi));
}

}  // namespace moe

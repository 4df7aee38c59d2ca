// kv_decode.cuh — E2M1 codes back to numbers, for the kernels that read the cache.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace nvfp4 {

// Two E2M1 codes (one byte, element 0 in the low nibble) -> two fp16, exact.
__device__ __forceinline__ uint32_t decode_e2m1x2_f16(uint32_t byte) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
        : "=r"(r)
        : "r"(byte));
    return r;
}
// Eight codes (element 0 in the lowest nibble) -> four fp16 pairs, exact.
__device__ __forceinline__ void decode_e2m1x8_f16(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// A UE4M3 scale byte -> the fp16 pair (s, s), exact.
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t byte) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\t"
        "cvt.u16.u32 h, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
        : "=r"(r)
        : "r"(byte * 0x0101u));
    return r;
}

// Two scale bytes (the low 16 bits) -> the fp16 pair (s0, s1), or (s0, s0) and (s1, s1); exact.
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t bytes) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\t"
        "cvt.u16.u32 h, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
        : "=r"(r)
        : "r"(bytes));
    return r;
}
__device__ __forceinline__ void scale2_f16x2(uint32_t bytes, uint32_t &s0, uint32_t &s1) {
    const uint32_t r = scales_f16x2(bytes);
    s0 = __byte_perm(r, r, 0x1010);
    s1 = __byte_perm(r, r, 0x3232);
}
// The power of two that brings a row whose largest magnitude is `top` to [2^14, 2^15), so that bf16
// becomes fp16 without losing a bit that matters; 1 for rows of zeros, infinities or NaN.  Its
// inverse (*inverse) is a normal number.
__device__ __forceinline__ float f16_row_factor(float top, float *inverse) {
    const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    const int sh = (top > 0.0f && top < INFINITY) ? min(max(14 - ex, -113), 126) : 0;
    *inverse = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
    return __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
}

// A row's score factor: the scale times the inverse, held within fp32's normal numbers (0 and infinity times a
// score that is infinite or 0 would be NaN).
__device__ __forceinline__ float score_factor(float scale, float inverse) {
    return fminf(fmaxf(scale * inverse, 1.17549435e-38f), 3.40282347e38f);
}

// Cached values take fp16 weights of up to 2^8 (what a score may outgrow its row's reference by).  Times 2^7 they
// still fit (2^15), and a weight below 2^-32 of the reference's, not 2^-25, rounds to none: over 2^20 keys with
// next to no weight each, what is lost is 2^-12 of the largest value at most, not 2^-5.  l and O carry the factor
// alike, and the division takes it out.
constexpr float kF16WeightBits = 7.0f;

}  // namespace nvfp4

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
__device__ __forceinline__ void decode_e2m1x8(uint32_t codes, float (&y)[8]) {
    uint32_t h[4];
    decode_e2m1x8_f16(codes, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        y[2 * j] = f.x;
        y[2 * j + 1] = f.y;
    }
}

}  // namespace nvfp4

// The 4-bit rows of a cache. A value is an e2m1 number (1 sign, 2 exponent
// and 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times the e4m3 scale that it
// shares with its 15 neighbours: 2 + 4 significant bits at most, exponents
// -10 to 11, so the product is exact in bf16 and in fp16.
//
// A pool holds, for a block and a KV head, records of 8 tokens: 8 rows of d / 2
// bytes of codes (the even element in the low four bits), then 8 rows of d / 16
// bytes of scales. A record is 9 d / 2 bytes, a multiple of 16 bytes for every
// d here, so that any run of 8-token groups of a block is one bulk copy.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace sp {

constexpr int kFp4Group = 16;             // elements of a scale
constexpr int kFp4Rows = 8;               // tokens of a record
constexpr uint32_t kFp4NoNumber = 0x7f;   // the e4m3 NaN

__host__ __device__ constexpr int fp4_record(int d) { return 9 * d / 2; }
__host__ __device__ constexpr int fp4_codes(int d) { return 4 * d; }   // bytes of codes in a record

__device__ __forceinline__ bool scale_is_nan(uint32_t byte) { return (byte & 0x7f) == kFp4NoNumber; }

// The four bytes of w: two e2m1 numbers each (low four bits first) as fp16.
__device__ __forceinline__ void fp4_unpack(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

// Two e4m3 numbers (the low 16 bits, low byte first) as fp16.
__device__ __forceinline__ uint32_t fp8_unpack(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\t"
        "mov.b32 {x, y}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, x;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}

// a * b in fp16, both halves (exact for a number and its scale).
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two fp32 values to the nearest e2m1 numbers (ties to the even code, at most
// 6), x in the low four bits.
__device__ __forceinline__ uint32_t fp4_pack2(float x, float y) {
    uint32_t r;
    asm("{\n\t.reg .b8 c;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\t"
        "cvt.u32.u8 %0, c;\n\t}"
        : "=r"(r)
        : "f"(x), "f"(y));
    return r;
}

// Nearest e4m3 number (ties to even, at most 448) of x >= 0.
__device__ __forceinline__ uint32_t fp8_pack(float x) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 c, %1, %2;\n\t"
        "cvt.u32.u16 %0, c;\n\t}"
        : "=r"(r)
        : "f"(0.0f), "f"(x));
    return r;
}

}  // namespace sp

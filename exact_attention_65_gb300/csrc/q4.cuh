// The 4-bit paged cache's format.
//
// Groups of 16 channels of a row share an e4m3 scale s, a channel is an e2m1
// code (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign), and the value is code * s
// times the tensor's own fp32 scale. A code has 2 significant bits and s has 4:
// code * s has at most 6 and lies within 2^-10 .. 2688, so it is exact in fp16
// and in bf16 and a product with it loses nothing that a 16-bit cache keeps.
// Scales are not negative; NaN stands for a group that held no number.
//
// A pool is [num_pages, h_kv, page_size * 9 d / 16] bytes. The block of a page
// and head is contiguous: page_size rows of d / 2 bytes of codes (channel 2 i in
// the low half of byte i), then page_size rows of d / 16 bytes of scales. Its
// parts begin at multiples of 16 bytes, as pages hold a multiple of 16 rows.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace exattn {

// Bytes of one row of one head, and where a page's scales begin.
__host__ __device__ constexpr int q4_code_bytes(int d) { return d / 2; }
__host__ __device__ constexpr int q4_scale_bytes(int d) { return d / 16; }
__host__ __device__ constexpr int64_t q4_block_bytes(int64_t page_size, int d) {
    return page_size * (q4_code_bytes(d) + q4_scale_bytes(d));
}

// Four bytes of codes as four pairs of fp16, byte i in r[i] (low code in the low half).
__device__ __forceinline__ void q4_codes_f16(uint32_t codes, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(codes));
}

// The scales in the low two bytes of s as a pair of fp16 (exact).
__device__ __forceinline__ uint32_t q4_scales_f16(uint32_t s) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(s));
    return r;
}

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Both halves at least 0; NaN becomes 0.
__device__ __forceinline__ uint32_t h2_max0(uint32_t a) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0u));
    return r;
}

// Four scale bytes: not 0 if one of them is NaN.
__device__ __forceinline__ uint32_t q4_scales_nan(uint32_t s) { return ((s & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Both halves of a pair of fp16 as fp32.
__device__ __forceinline__ float2 h2_float2(uint32_t x) {
    float2 r;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(x));
    return r;
}

// A scale byte from an fp32 value: nearest, ties to even, at most 448; NaN stays.
__device__ __forceinline__ uint32_t q4_scale_byte(float s) {
    uint32_t r;
    asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %1, %2;\n\tcvt.u32.u16 %0, x;\n\t}"
        : "=r"(r)
        : "f"(0.0f), "f"(s));
    return r & 0xffu;
}

// Two codes in a byte, lo in its low half: nearest, ties to even, at most 6.
__device__ __forceinline__ uint32_t q4_code_byte(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 x, z;\n\tcvt.rn.satfinite.e2m1x2.f32 x, %1, %2;\n\tmov.b32 %0, {x, 0, 0, 0};\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Both halves of a pair of fp32 negated.
__device__ __forceinline__ uint64_t f2_neg(uint64_t x) { return x ^ 0x8000000080000000ull; }

// 16 bytes at a 16-byte-aligned shared-memory address.
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

}  // namespace exattn

// Device helpers of the 4-bit cache: the two number formats, and where a row
// lies in the pool.
//
// A value is code * scale: the code one e2m1 (sign, two exponent bits, one
// mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), the scale one e4m3 per 16 dims.
// Their product has at most 2 + 4 significant bits and lies in
// [2^-10, 2688], so f16 and bf16 both hold it exactly: whatever reads the
// cache works on the stored values without a rounding of its own.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "attn_internal.h"

namespace attn {
namespace kv4 {

// Four code bytes (dims 2i, 2i + 1 in byte i) -> four f16 pairs.
__device__ __forceinline__ void codes_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
// Two e4m3 scales (low byte, high byte) -> an f16 pair (exact).
__device__ __forceinline__ uint32_t scales_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// (a, b) -> code bytes, round to nearest even, saturating: a in the low nibble.
__device__ __forceinline__ uint32_t code_pair(float a, float b) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
        "mov.b32 %0, {t, 0, 0, 0};\n\t}"
        : "=r"(r) : "f"(a), "f"(b));
    return r;
}
// The e4m3 byte nearest to x >= 0 (448 at most; NaN stays NaN).
__device__ __forceinline__ uint32_t scale_byte(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xFFu;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Byte offset of the 16 tokens that hold row `row` of (page, K/V `half`, KV
// head g).  Within them, token row % 16 has its codes at (row % 16) * D / 2
// and its scales at 8 D + (row % 16) * D / 16.
__device__ __forceinline__ int64_t sub_offset(int64_t page, int half, int Hkv, int g, int P, int row, int sub_bytes) {
    return (((page * 2 + half) * Hkv + g) * (P / kKv4Tokens) + row / kKv4Tokens) * sub_bytes;
}

}  // namespace kv4
}  // namespace attn

// The 4-bit KV format: E2M1 codes with one E4M3 scale for 16 values.
//
// A pool row holds one token's K (or V) of every KV head.  Heads are kept in
// blocks of four (the last may hold fewer): a block is its heads' codes
// (d / 2 bytes each, element 2i in the low half of byte i), then its heads'
// scales (d / 16 bytes each).  Any run of whole blocks is contiguous, so a
// streaming piece of 4 or 8 heads is one copy, codes start on 16-byte
// boundaries and a head's scales on d / 16-byte ones.  Rows are padded to a
// multiple of 16 bytes.
//
// value = tensor scale * sf * e2m1.  sf * e2m1 has at most 1 + 3 + 1 bits
// after its leading one and lies in [2^-10, 2688] or is 0: f16 holds it
// exactly, so the kernels' only rounding of a cached value is the one made
// when it was stored.
#pragma once

#include "device_common.cuh"

namespace sgldev {

// Attention over a 4-bit pool holds the softmax weights as f16: 2^kPShift times
// exp2(score - maximum), the maximum being up to 8 too low.
constexpr float kPShift = 7.f;

// bytes of one head's codes and scales, of a block of `n` <= 4 heads, and
// the offset of head h's block (every block before it is full)
__host__ __device__ constexpr int fp4_head_bytes(int d) { return d / 2 + d / 16; }
__host__ __device__ constexpr int fp4_row_bytes(int hkv, int d) { return (hkv * fp4_head_bytes(d) + 15) / 16 * 16; }
// offset of head h's codes / scales within a row of hkv heads
__host__ __device__ __forceinline__ int fp4_code_off(int h, int d) {
    return (h >> 2) * 4 * fp4_head_bytes(d) + (h & 3) * (d / 2);
}
__host__ __device__ __forceinline__ int fp4_scale_off(int h, int hkv, int d) {
    const int n = hkv - (h & ~3) < 4 ? hkv - (h & ~3) : 4;
    return (h >> 2) * 4 * fp4_head_bytes(d) + n * (d / 2) + (h & 3) * (d / 16);
}

// E4M3 code of x, nearest even, saturated at 448 (NaN kept)
__device__ __forceinline__ uint32_t e4m3_of(float x) {
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(x));
    return h & 0xffu;
}
// the value of an E4M3 code (exact)
__device__ __forceinline__ float e4m3_value(uint32_t code) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}
// E2M1 codes of eight values, nearest even, saturated at 6: element i in
// bits 4i .. 4i + 3
__device__ __forceinline__ uint32_t e2m1x8_of(const float* x) {
    uint32_t w;
    asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(w)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return w;
}
// Eight E2M1 codes (one word) as four f16x2 words (exact), in order.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t* h) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b;\n cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Two E4M3 scales (the low 16 bits) as an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
    return h;
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

}  // namespace sgldev

// fp4.cuh -- the 4-bit form: a row of values as e2m1 codes (two a byte, the
// first in the low half), an e4m3 byte for each block of 16 of them and one fp32
// scale:  value = scale * e4m3(block) * e2m1(code).
//
// A code has two significant bits and a block's scale four, so their product has
// six, between 2^-10 and 2688: exact in fp16, in bf16 and in fp32.  Kernels fold
// the block's scale into the 16-bit operand and leave the row's to their fp32
// epilogue, so the form adds no rounding to that of its codes.
#pragma once

#include "fp8w_device.cuh"

namespace fp8w {

// 8 codes (one word) -> four f16x2, in order.  The conversion runs at 48 lanes a
// cycle and SM (measured); placing the bits by shifts and masks at half of that.
// One statement a byte: all four out of one unpacking take a move each.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t& p0, uint32_t& p1, uint32_t& p2, uint32_t& p3) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(p0) : "r"(w));
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(p1) : "r"(w));
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(p2) : "r"(w));
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(p3) : "r"(w));
}

// Eight fp32 values -> their nearest-even, saturated codes in order.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&f)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return w;
}
__device__ __forceinline__ uint16_t f32x4_to_e2m1(float f0, float f1, float f2, float f3) {
    uint16_t h;
    asm("{\n\t.reg .b8 a, b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "mov.b16 %0, {a, b};\n\t}"
        : "=h"(h)
        : "f"(f0), "f"(f1), "f"(f2), "f"(f3));
    return h;
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Scales of two blocks as a factor of decoded codes (fp16 pairs).
__device__ __forceinline__ uint32_t block_pair_f16(uint32_t two) { return e4m3x2_to_f16x2(static_cast<uint16_t>(two)); }
__device__ __forceinline__ uint32_t both_lo(uint32_t pair) { return __byte_perm(pair, pair, 0x1010); }
__device__ __forceinline__ uint32_t both_hi(uint32_t pair) { return __byte_perm(pair, pair, 0x3232); }

// fp16 pair -> bf16 pair (exact where the values have 8 significant bits), by
// fp32: two instructions of the FMA pipe and one of the ALU's, which the codes'
// conversion keeps busy.  (Moving the exponent's bits by a shift and two masks, and
// 2^112 into the block's factor: 32 tokens on 14336 x 4096 20.2 us when this took 17.7,
// a prompt 204 against 195, attention of chunks 887 against 818.)
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t p) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\t.reg .f32 x, y;\n\t"
        "mov.b32 {a, b}, %1;\n\t"
        "cvt.f32.f16 x, a;\n\tcvt.f32.f16 y, b;\n\t"
        "cvt.rn.bf16x2.f32 %0, y, x;\n\t}"
        : "=r"(r)
        : "r"(p));
    return r;
}

// Eight codes as 16-bit operands, in order, times their block's scale (both halves
// of `factor`).
template <bool kBf16>
__device__ __forceinline__ void fp4_operands(uint32_t w, uint32_t factor, uint32_t* v) {
    e2m1x8_to_f16x2(w, v[0], v[1], v[2], v[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = f16x2_mul(v[e], factor);
        if constexpr (kBf16) v[e] = f16x2_to_bf16x2(v[e]);
    }
}

// The quantiser's rule, all steps in fp32 with one rounding each:
//   scale = max(amax * (1 / 2688), 2^-126), 1 where amax is 0   (2688 = 6 * 448)
//   y     = x * (1 / scale)
//   block = e4m3(max over the block of |y| * (1 / 6)), nearest even
//   code  = e2m1(y * (1 / block)), nearest even, saturated; 0 where block is 0
// The floor keeps 1 / scale finite.
__device__ __forceinline__ float fp4_scale(float amax) {
    return amax == 0.0f ? 1.0f : fmaxf(__fmul_rn(amax, 1.0f / 2688.0f), 1.17549435e-38f);
}
__device__ __forceinline__ uint32_t fp4_block(float ymax) {  // the byte
    return f32x2_to_e4m3x2(__fmul_rn(ymax, 1.0f / 6.0f), 0.0f) & 0xFFu;
}
__device__ __forceinline__ float fp4_block_inverse(uint32_t byte) {
    return byte == 0u ? 0.0f : __frcp_rn(f16_lo_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(byte))));
}

}  // namespace fp8w

// The 4-bit KV format shared by the kernels that write and read it: the row
// layout of a pool, and the conversions between codes and numbers.
//
// A pool row holds one token.  Its Hkv heads lie in groups of gs (the largest
// power of two up to 8 that divides Hkv); a group is
//   gs * d/2 bytes   E2M1 codes, two to a byte (element 2j in the low nibble)
//   gs * d/16 bytes  E4M3 scales, one per head and block of 16 elements
// padded to a multiple of 16 bytes, so that a group's rows can be moved with
// bulk copies.  The heads a decode CTA reads together are one group: with at
// most 8 KV heads a row is one group and a 16-token page one contiguous run.
// Element x of block b of head h reads as value(code) * value(scale_b) * g_h,
// g the caller's fp32 scale of the head; the first product has at most six
// significant bits and lies between 2^-10 and 2688, so it is exact in f16.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace pa {

struct Fp4Layout {
    int gs;            // heads of a group
    int groups;
    int code_bytes;    // of a group
    int group_bytes;   // with scales and padding
    int row_bytes;
};

__host__ __device__ inline Fp4Layout fp4_layout(int hkv, int d) {
    Fp4Layout l;
    l.gs = 8;
    while (hkv % l.gs != 0) l.gs >>= 1;
    l.groups = hkv / l.gs;
    l.code_bytes = l.gs * d / 2;
    l.group_bytes = (l.code_bytes + l.gs * d / 16 + 15) / 16 * 16;
    l.row_bytes = l.groups * l.group_bytes;
    return l;
}

#ifdef __CUDACC__

// Eight E2M1 codes (a 32-bit word, element 2j in the low nibble of byte j) to
// eight f16.  Measured with the multiply by the block scale that follows: 84
// elements per clock and SM, against 45 to 52 for forms made of shifts and
// masks; HBM delivers 42 (9/16 byte each).
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}

// Two E4M3 codes (the low 16 bits) to two f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(two_codes));
    return r;
}

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The factor that takes raw scores to log2 units, the head's K scale in it.  A
// scale of zero (an all-zero head's) would make 0 * -inf = NaN of the masked
// scores; the smallest normal number, 2^-126, leaves them -inf and every other
// score, at most 2^35 raw (128 products of 2688 and 65504), zero to within
// 2^-91.  A NaN stays one.
__device__ __forceinline__ float fp4_score_scale(float scale_log2, float k_scale) {
    const float s = scale_log2 * k_scale;
    return s < 1.17549435e-38f ? 1.17549435e-38f : s;
}

// One f16 of a pair in both halves.
__device__ __forceinline__ uint32_t f16_dup_lo(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t f16_dup_hi(uint32_t x) { return __byte_perm(x, x, 0x3232); }

#endif  // __CUDACC__

}  // namespace pa

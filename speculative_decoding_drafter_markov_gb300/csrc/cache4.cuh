// cache4.cuh -- a cache of 4 bits per element (include/dspark.h has the format): scale
// bytes, codes and where they stand.
#pragma once

#include "common.cuh"

namespace dspark {
namespace cache4 {

constexpr int kGroup = 16;              // elements of a scale
constexpr unsigned kNoNumbers = 255;    // scale byte of 16 elements that are NaN

// bytes of a page of one head, and of its codes
__host__ __device__ __forceinline__ long long page_bytes(int page, int D) { return (long long)page * D / 16 * 9; }
__host__ __device__ __forceinline__ long long code_bytes(int page, int D) { return (long long)page * (D / 2); }

// s(b) = 2^(b / 8 - 16) (1 + b % 8 / 8): byte b is the exponent's low bits and three bits of
// the fraction, so a shift and an addition make it a float
__device__ __forceinline__ float scale_of(unsigned b) {
    return b == kNoNumbers ? __uint_as_float(0x7fc00000u) : __uint_as_float((b + (111u << 3)) << 20);
}

// where element e of 8 stands in their four bytes, as a shift
__device__ __forceinline__ int code_shift(int e) { return 4 * (4 * (e & 1) + (e >> 1)); }

// The scale byte of 16 elements whose largest magnitude is `most`: the quotient cut to
// three bits of fraction is s(b) or the one below the nearest; most is compared
// with 7 times the middle of s(b) and s(b + 1), a product of five bits and three, which
// is exact.
__device__ __forceinline__ unsigned scale_byte(float most) {
    if (!(most < INFINITY)) return kNoNumbers;
    const float want = fminf(fmaxf(most * (1.f / 7.f), 0x1p-16f), 57344.f);
    const unsigned cut = __float_as_uint(want) >> 20, b = cut - (111u << 3);
    const float middle7 = 7.f * __uint_as_float((cut << 20) | (1u << 19));
    const unsigned up = most > middle7 || (most == middle7 && (b & 1u));
    return min(b + up, 254u);
}

// n = x / s rounded to the nearest whole number (halfway: the even one), within -7 .. 7,
// exactly, for x of float: the product with 1 / s may be off in its last bits, so the
// whole number below is settled by comparing x with (n + 1/2) s, which is exact (four
// bits and four)
__device__ __forceinline__ float whole_of(float x, float s, float inv) {
    const float a = fabsf(x), low = fminf(floorf(a * inv), 7.f), half = (low + 0.5f) * s;
    const float n = low + ((a > half || (a == half && ((int)low & 1))) ? 1.f : 0.f);
    return copysignf(fminf(n, 7.f), x);
}
// The same for x of bf16, as the float 1.5 2^23 + 8 + n (its lowest byte is the code): x / s is a
// quotient of eight bits and four, which is halfway between two whole numbers or at
// least 2^-11 away (|x / s| between 1/4 and 16: a multiple of 2^-6 / 30 off any odd half).
// Rounded to a multiple of 2^-14 it is on the right side, whatever the product with 1 / s
// loses.  It is within -7.44 .. 7.44 unless the scale is the largest there is.
__device__ __forceinline__ float coded_bf16(float x, float inv) {
    return __fadd_rn(__fmaf_rn(x, inv, 768.f), 12582920.f - 768.f);  // 768 = 1.5 2^9
}
constexpr float kMostHeld = 7.f * 57344.f;

// ---------------------------------------------------------------- two values at a time
// A code word has elements 2 p and 2 p + 1 of eight in nibble p of its halves, so a shift and a
// mask with an exponent make two numbers of it, and one or two operations the values.  (That way
// from 4 bits to fp16, and an order of the elements that serves it, are published: Kim et al., "Who
// Says Elephants Can't Run", arXiv 2211.10017; the constants follow from the formats.)

// (x & mask) | bits, in one instruction
template <uint32_t kMask, uint32_t kBits>
__device__ __forceinline__ uint32_t mask_or(uint32_t x) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(kMask), "r"(kBits));
    return y;
}
// s(b) twice in bf16, b <= 254: (b + 888) << 4 are its bits
__device__ __forceinline__ uint32_t bf16_scales(uint32_t b) { return b * 0x00100010u + 0x37803780u; }
// -136 s: 17 s 8, eight bits, so it is exact
__device__ __forceinline__ uint32_t bf16_offset(uint32_t s) {
    uint32_t y;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(s), "r"(0xc308c308u));
    return y;
}
// values of nibble p in bf16: 128 + (n + 8) by its bits, times s, minus 136 s
__device__ __forceinline__ uint32_t bf16_of(uint32_t word, int p, uint32_t s, uint32_t off) {
    const uint32_t v = mask_or<0x000f000fu, 0x43004300u>(word >> (4 * p));
    uint32_t y;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(v), "r"(s), "r"(off));
    return y;
}
// s(b) / 8, b <= 254.  Eighths of values, 2^-19 to 50176, are exact in fp16.
__device__ __forceinline__ float eighth_of(uint32_t b) { return __uint_as_float(b * 0x00100000u + (108u << 23)); }
// eighths of the values of nibble 0 (odd: 1) in fp16, s: s / 8 twice: 1024 + (n + 8), or
// 1024 + 16 (n + 8) one nibble up, to n, times s
__device__ __forceinline__ uint32_t half_of(uint32_t word, int odd, uint32_t s) {
    uint32_t n, y;
    if (odd) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(n) : "r"(mask_or<0x00f000f0u, 0x64006400u>(word)), "r"(0x2c002c00u), "r"(0xd480d480u));  // 1 / 16, -72
    else asm("add.rn.f16x2 %0, %1, %2;" : "=r"(n) : "r"(mask_or<0x000f000fu, 0x64006400u>(word)), "r"(0xe408e408u));  // -1032
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(n), "r"(s));
    return y;
}

}  // namespace cache4
}  // namespace dspark

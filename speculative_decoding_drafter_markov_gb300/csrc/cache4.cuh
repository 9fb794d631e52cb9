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
// and for x of bf16: x / s is a quotient of eight bits and four, which is halfway between
// two whole numbers or at least 2^-11 away (|x / s| between 1/4 and 16: a multiple
// of 2^-6 / 30 off any odd half).  Rounded to a multiple of 2^-14 it is on the right side,
// whatever the product with 1 / s loses.
__device__ __forceinline__ float whole_of_bf16(float x, float inv) {
    const float t = __fadd_rn(__fmaf_rn(x, inv, 768.f), -768.f);  // 768 = 1.5 2^9
    return fminf(fmaxf(__fadd_rn(__fadd_rn(t, 12582912.f), -12582912.f), -7.f), 7.f);  // 1.5 2^23
}

}  // namespace cache4
}  // namespace dspark

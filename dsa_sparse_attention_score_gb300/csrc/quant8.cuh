// quant8.cuh -- the 8-bit latent row: e4m3 codes under one power-of-two scale.
//
// A row x (512 latent values and, with a tail, 64 rotated ones) is held as
//     E     = the least integer in [-40, 119] with max |x| <= 448 * 2^E,
//     code  = e4m3(x / 2^E)                        for the latent values,
//     hi    = e4m3(r / 2^E), lo = e4m3(r / 2^E - hi)  for a tail value r,
// every conversion rounding to nearest even.  2^E is a power of two, so the
// division is exact and each code is off by at most half an e4m3 step: 2^-4
// of its value down to 2^-6 * 2^E, 2^-10 * 2^E below.  The tail keeps a
// remainder because its products are not averaged over 512 terms: hi + lo is
// within 2^-8 of the value (or 2^-10 * 2^E).
//
// One scale per row, not one per group of columns: e4m3 carries four bits of
// exponent of its own, so finer scales would only help values below 2^-14 of
// the row's largest, and a per-row scale leaves every contraction over the
// row's columns a plain 8-bit matrix product (the tensor cores read the codes
// as they are).  E is kept above -40 so that 1 / 2^E and its products stay
// far from the float32 range's ends, and below 120 so that 448 * 2^E is
// finite; a row holding NaN or infinity gets the scale NaN and codes 0.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace dsa {

constexpr int kQ8MinExp = -40, kQ8MaxExp = 119;

// 2^n for -126 <= n <= 127.
__device__ __forceinline__ float exp2_int(int n) { return __int_as_float((n + 127) << 23); }

// E of values whose largest magnitude is top (finite): 448 = 1.75 * 2^8.
__device__ __forceinline__ int q8_exponent(float top, int least = kQ8MinExp) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 127 - ((b & 0x7FFFFFu) > 0x600000u ? 7 : 8);
    return min(max(e, least), kQ8MaxExp);
}

// Two e4m3 codes, lo_elem in bits 0..7.
__device__ __forceinline__ uint32_t e4m3x2(float lo_elem, float hi_elem) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi_elem), "f"(lo_elem));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2(__half2 v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&v)));
    return r;
}
// The same in e5m2, whose smallest step is 2^-16 against e4m3's 2^-9.
__device__ __forceinline__ uint32_t e5m2x2(__half2 v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&v)));
    return r;
}
// The values of two e4m3 codes (bits 0..7 first), exact in fp16.
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return *reinterpret_cast<const __half2 *>(&h);
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) { return __half22float2(e4m3x2_to_half2(codes)); }

}  // namespace dsa

// rope.cuh -- the rotation angle of a (position, pair).
#pragma once

#include <stdint.h>

namespace dsa {

struct DevRope {
    const double *inv_freq;   // device [rot_dim / 2], radians per position
    int rot_dim;              // values rotated (even)
    int interleaved;          // pairs (2j, 2j+1), else (j, j + rot_dim / 2)
    float scale;              // factor on the rotated values
    int inverse;              // turn by -angle
};

// scale * (cos, sin) of pos * inv_freq.
//
// A 32-bit angle would be off by 0.03 radians at position 10^6, and 64-bit
// floating point runs at a sixteenth of a lane per cycle and SM partition here
// (one row per warp spent more time on its angle than on its bytes), so the
// angle is formed in integers, as a fraction of a turn in units of 2^-64:
//     inv_freq = m 2^(e - 1075), m of 53 bits
//     F        = frac(inv_freq / 2 pi) 2^64 = m C 2^(e - 1075) mod 2^64,  C = 2^64 / 2 pi
//     turn     = pos F mod 2^64.
// Whole turns drop out by wrapping.  C and F are cut to their units, so F is
// off by less than |inv_freq| + 1 of them and the turn by less than
// (|inv_freq| + 1) |pos| 2^-64; the fraction, in [-1/2, 1/2), is cut to 2^-32.
// float32 holds 24 bits of it, and a turn by the rest follows the sine and
// cosine: they are off by 8e-8 at most, 1.1e-7 without it.  Either sign; a
// frequency that is NaN or infinite gives NaN.
__device__ __forceinline__ float2 rope_cos_sin(int32_t pos, double inv_freq, float scale, int inverse) {
    const uint64_t bits = (uint64_t)__double_as_longlong(inv_freq);
    const int exponent = (int)((bits >> 52) & 0x7FF), shift = 1075 - exponent;
    if (exponent == 0x7FF) scale = __int_as_float(0x7FC00000);
    const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
    constexpr uint64_t C = 0x28BE60DB9391054Aull;             // floor(2^64 / (2 pi))
    const uint64_t lo = m * C, hi = __umul64hi(m, C);
    uint64_t F = 0;
    if (shift <= 0) F = shift > -64 ? lo << -shift : 0;
    else if (shift < 64) F = (lo >> shift) | (hi << (64 - shift));
    else if (shift < 128) F = hi >> (shift - 64);
    if (bits >> 63) F = ~F + 1;
    const uint64_t turn = F * (uint64_t)(int64_t)pos;
    const int32_t frac = (int32_t)(turn >> 32);
    const float near = (float)frac;
    float s, c;
    sincospif(near * 0x1p-31f, &s, &c);
    // what the conversion left out, at most 2^6 units: sin(a + d) = sin a + d cos a
    const float d = (float)(frac - __float2int_rz(near)) * (6.2831853f * 0x1p-32f), s0 = s;
    s = fmaf(c, d, s);
    c = fmaf(-s0, d, c);
    return make_float2(c * scale, inverse ? -s * scale : s * scale);
}

}  // namespace dsa

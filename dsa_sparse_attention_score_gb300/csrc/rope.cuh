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

// scale * (cos, sin) of pos * inv_freq.  The angle is formed and reduced to a
// fraction of a turn in 64 bits -- at position 10^6 a 32-bit product would be
// off by 0.03 radians -- and the fraction, below 1/2, rounded once to 32.
__device__ __forceinline__ float2 rope_cos_sin(int32_t pos, double inv_freq, float scale, int inverse) {
    double turns = (double)pos * inv_freq * 0.15915494309189533576888;   // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    return make_float2(c * scale, inverse ? -s * scale : s * scale);
}

}  // namespace dsa

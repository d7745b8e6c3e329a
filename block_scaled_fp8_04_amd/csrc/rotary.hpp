// rotary.hpp - a position's angles and a pair's turn on gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bfp8 {

// amplitude * (cos, sin) of position * inv_freq.  A far position's angle has more digits than fp32
// holds behind its whole turns: it is formed in 64 bits and reduced to half a turn there.  With inv_freq
// up to 1 the angle is off by 2^-25.9 of a turn at most for positions below 2^24 (2^-26 of it the last
// rounding, to fp32), by 2^-22.9 for any 32-bit one (three roundings of 2^28.4 turns in 64 bits besides).
__device__ __forceinline__ float2 rotary(int32_t position, float inv_freq, float amplitude) {
    const double turns = (double)position * (double)inv_freq * 0.15915494309189535;
    const float half_turns = 2.f * (float)(turns - __builtin_rint(turns));
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * amplitude, s * amplitude);
}

// (a, b) turned by an angle's cosine and sine.
__device__ __forceinline__ void turn(float& a, float& b, const float2 cs) {
    const float x = a;
    a = __builtin_fmaf(x, cs.x, -b * cs.y);
    b = __builtin_fmaf(x, cs.y, b * cs.x);
}

}  // namespace bfp8

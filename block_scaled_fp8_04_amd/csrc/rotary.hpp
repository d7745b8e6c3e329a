// rotary.hpp - a position's angles on gfx950.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bfp8 {

// amplitude * (cos, sin) of position * inv_freq.  A far position's angle has more digits than fp32
// holds behind its whole turns: it is formed in 64 bits and reduced to half a turn there, 2^-28 of a
// turn off at most for any 32-bit position.
__device__ __forceinline__ float2 rotary(int32_t position, float inv_freq, float amplitude) {
    const double turns = (double)position * (double)inv_freq * 0.15915494309189535;
    const float half_turns = 2.f * (float)(turns - __builtin_rint(turns));
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * amplitude, s * amplitude);
}

}  // namespace bfp8

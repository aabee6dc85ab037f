// Rotation angles of integer positions.
#pragma once

#include <stdint.h>

namespace qa {

// cos/sin of 2 pi pos (t_hi + t_lo), 0 <= pos < 2^18, t a frequency in turns
// (t_hi = t rounded to fp32, t_lo the rounding of the rest).  pos t_hi is
// carried exactly, as its fp32 rounding and the FMA residual; taking off the
// whole turns of the rounding is exact too, so the fraction is within about
// 2^-24 of a turn of the true one.  Then the hardware sine and cosine, within
// 2^-20.5 on [-pi, pi]: results are rounded to bf16, whose half step is 2^-9
// or more of the pair.
__device__ __forceinline__ void sincos_turns(int pos, float t_hi, float t_lo, float *s, float *c) {
    const float p = (float)pos;
    const float turns = p * t_hi;
    const float rest = fmaf(p, t_hi, -turns) + p * t_lo;
    const float a = 6.2831853071795865f * ((turns - rintf(turns)) + rest);
    *s = __sinf(a);
    *c = __cosf(a);
}

}  // namespace qa

// Rotation angles of integer positions.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __CUDACC__
#define QA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define QA_HOST_DEVICE inline
#endif

namespace qa {

// pos (t_hi + t_lo) less its whole turns, in [-1/2, 1/2]: 0 <= pos < 2^18, t a
// frequency in turns, at most 1 / 2 pi (t_hi = t rounded to fp32, t_lo the
// rounding of the rest).  pos t_hi is carried exactly, as its fp32 rounding
// and the FMA residual; taking off the whole turns of the rounding is exact
// too, so the fraction is within 2^-24 of a turn of the true one.  The
// residual, up to 2^-9 of a turn, can take it past half a turn: off again.
QA_HOST_DEVICE float turn_fraction(int pos, float t_hi, float t_lo) {
    const float p = (float)pos;
#ifdef __CUDA_ARCH__
    const float turns = __fmul_rn(p, t_hi);  // rounded by itself: in an FMA the residual would count twice
#else
    const float turns = p * t_hi;
#endif
    const float rest = fmaf(p, t_lo, fmaf(p, t_hi, -turns));
    const float f = (turns - rintf(turns)) + rest;
    return f - rintf(f);
}

#ifdef __CUDACC__
// cos/sin of 2 pi pos (t_hi + t_lo).  The hardware sine and cosine are within
// 2^-20.5 on [-pi, pi], so a rotated value is within about that of the size
// of its pair.  Results are rounded to bf16, whose half step is 2^-9 of the
// value itself: it hides this error unless the rotation cancels to less than
// 2^-11 of the pair.
__device__ __forceinline__ void sincos_turns(int pos, float t_hi, float t_lo, float *s, float *c) {
    const float a = 6.2831853071795865f * turn_fraction(pos, t_hi, t_lo);
    *s = __sinf(a);
    *c = __cosf(a);
}
#endif

}  // namespace qa

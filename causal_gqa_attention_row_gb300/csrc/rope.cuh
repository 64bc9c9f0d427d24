// rope.cuh -- sine and cosine of a rotary angle (position times frequency),
// reduced accurately: shared by the rotation, append and q/k row kernels.
#pragma once

#include <cuda_runtime.h>

namespace gqa {

// 2*pi split into a double and the double nearest to its remainder (Cody and
// Waite's reduction): a - n*HI - n*LO keeps ~1e-15 rad for |n| < 2^20.
constexpr double kTwoPiHi = 6.283185307179586;
constexpr double kTwoPiLo = 2.4492935982947064e-16;
constexpr double kInvTwoPi = 0.15915494309189535;

__device__ __forceinline__ void rope_cos_sin(double pos, double w, float* c, float* s) {
  const double a = pos * w;
  const double n = rint(a * kInvTwoPi);
  const double r = fma(-n, kTwoPiLo, fma(-n, kTwoPiHi, a));
  sincosf((float)r, s, c);
}

// The same in fp32 arithmetic, which this GPU runs far faster than fp64, for
// |pos| < 2^24 (the position exact in a float). The frequency comes as a float
// pair w_hi + w_lo within 2^-48 of the double; the product pos * w is formed
// without error in a_hi + e (Dekker and Kahan's two-product: one FMA gives the
// rounding error of pos * w_hi), and the reduction modulo 2*pi is Cody and
// Waite's with 2*pi as the sum of three floats, one FMA per part. The reduced
// angle is within ~3e-7 rad of the exact one (the fp64 form, which also rounds
// it to a float before sincosf, within ~1.2e-7).
constexpr float kTwoPiF1 = 6.2831854820251465f;       // the float nearest 2*pi
constexpr float kTwoPiF2 = -1.7484555314695172e-07f;  // ... nearest 2*pi - kTwoPiF1
constexpr float kTwoPiF3 = -6.8604980400235275e-15f;  // ... nearest what remains (4e-23 left)
constexpr float kInvTwoPiF = 0.15915493667125702f;

__device__ __forceinline__ void rope_cos_sin_f(int pos, float w_hi, float w_lo, double w, float* c, float* s) {
  if (pos >= (1 << 24) || pos <= -(1 << 24)) {  // not exact as a float
    rope_cos_sin((double)pos, w, c, s);
    return;
  }
  const float p = (float)pos;
  const float a_hi = p * w_hi;
  const float a_lo = fmaf(p, w_lo, fmaf(p, w_hi, -a_hi));  // the rounding error of p * w_hi, plus p * w_lo
  const float n = rintf(a_hi * kInvTwoPiF);
  float r = fmaf(-n, kTwoPiF1, a_hi);
  r = fmaf(-n, kTwoPiF2, r);
  r = fmaf(-n, kTwoPiF3, r);
  sincosf(r + a_lo, s, c);
}

// The same with the frequency given as the float pair alone.
__device__ __forceinline__ void rope_cos_sin_pair(int pos, float w_hi, float w_lo, float* c, float* s) {
  if (pos >= (1 << 24) || pos <= -(1 << 24))
    rope_cos_sin((double)pos, (double)w_hi + (double)w_lo, c, s);
  else
    rope_cos_sin_f(pos, w_hi, w_lo, 0.0, c, s);
}

}  // namespace gqa

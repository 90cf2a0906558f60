// Device helpers of the rotary positions: sines and cosines of a pair's angle, and its turn.
//
// Angles: the product is exact in 64 bits (24 + 24 bits of the factors), is turned into
// revolutions and loses its whole turns there, so that a position far along an axis is as exact
// as a near one; the rest is a Taylor polynomial on an eighth turn either way.
#pragma once

#include "attention_device.h"

namespace orbq {

__device__ __forceinline__ void sincos_revolutions(double rev, float* s, float* c) {
  const float f = static_cast<float>(rev - __builtin_rint(rev));  // [-1/2, 1/2]
  const float quarter = __builtin_rintf(4.0f * f);
  const float x = (f - 0.25f * quarter) * 6.28318530717958648f;   // [-pi/4, pi/4]
  const float x2 = x * x;
  // Taylor to x^9 and x^10: the next terms are below 2e-9 and 5e-10
  float sn = 2.7557319e-6f, cs = -2.7557319e-7f;
  sn = __builtin_fmaf(sn, x2, -1.9841270e-4f);
  sn = __builtin_fmaf(sn, x2, 8.3333333e-3f);
  sn = __builtin_fmaf(sn, x2, -1.6666667e-1f);
  sn = __builtin_fmaf(sn * x2, x, x);
  cs = __builtin_fmaf(cs, x2, 2.4801587e-5f);
  cs = __builtin_fmaf(cs, x2, -1.3888889e-3f);
  cs = __builtin_fmaf(cs, x2, 4.1666667e-2f);
  cs = __builtin_fmaf(cs, x2, -0.5f);
  cs = __builtin_fmaf(cs, x2, 1.0f);
  const int k = static_cast<int>(quarter) & 3;
  const float a = (k & 1) ? cs : sn, b = (k & 1) ? sn : cs;
  *s = (k & 2) ? -a : a;
  *c = ((k + 1) & 2) ? -b : b;
}

// A: RopeArgs or another that holds axes, ends, freqs and inverse as it does
template <class A> __device__ __forceinline__ void pair_sincos(const A& a, const float* pos, int pair, float* s, float* c) {
  int axis = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k) axis += (k < a.axes - 1 && pair >= a.ends[k]) ? 1 : 0;
  const double rev = static_cast<double>(pos[axis]) * static_cast<double>(a.freqs[pair]) * 0.15915494309189533577;
  sincos_revolutions(rev, s, c);
  if (a.inverse) *s = -*s;
}

// one rounding order for every form, so that strides and alignment do not change bits
__device__ __forceinline__ void turn(float a, float b, float s, float c, float* u, float* w) {
  *u = __builtin_fmaf(a, c, -(b * s));
  *w = __builtin_fmaf(a, s, b * c);
  // keeps the compiler from joining the sum with the rounding to f16 in one form and not in another
  asm("" : "+v"(*u), "+v"(*w));
}

}  // namespace orbq

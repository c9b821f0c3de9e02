// The angle of a rotary position, exact for far ones.
//
// pos x theta is needed modulo a turn.  In turns, theta / 2 pi is a fixed-point
// fraction of 64 bits, F, and pos F modulo 2^64 is an integer product: the error
// of the angle is |pos| 2^-64 turns from F (2^-40 of a turn at 16 million tokens)
// and 2^-32 of a turn from the final 32 bits.  (In float32 pos x theta itself has
// an error of 0.03 radians at a million tokens; in float64 the products run at a
// sixtieth of the float32 rate.)
#pragma once

#include <stdint.h>

namespace llattn {

// theta / 2 pi as a fraction of 2^64 (modulo 1); theta any finite float32 value.
__device__ __forceinline__ uint64_t rope_turns(float theta) {
  const uint32_t u = __float_as_uint(theta);
  const int e = (int)((u >> 23) & 255);
  const uint64_t m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);  // theta = m 2^-s
  const int s = 150 - (e ? e : 1);
  // m / 2 pi 2^40, from 1 / 2 pi = 0x.28be60db9391054a (7f09d5f4...)
  const uint64_t x = __umul64hi(m << 40, 0x28be60db9391054aull);
  const int sh = s - 24;
  const uint64_t f = sh >= 64 ? 0 : sh >= 0 ? x >> sh : sh > -64 ? x << -sh : 0;
  return (u >> 31) ? 0 - f : f;
}
// cos and sin of pos theta, F = rope_turns(theta)
__device__ __forceinline__ void rope_sincos(long long pos, uint64_t f, float& s, float& c) {
  const int32_t a = (int32_t)(((uint64_t)pos * f) >> 32);  // in units of 2^-32 turns, from -1/2 to 1/2
  sincospif((float)a * 4.656612873077393e-10f, &s, &c);     // 2^-31
}

// The same by the hardware's own sine, whose error on [-pi, pi] is 2^-21 and more: for
// results that are rounded to bf16, 2^-9 of their size.
__device__ __forceinline__ void rope_sincos_fast(long long pos, uint64_t f, float& s, float& c) {
  const int32_t a = (int32_t)(((uint64_t)pos * f) >> 32);
  const float x = (float)a * 1.4629180792671596e-9f;  // 2 pi 2^-32
  s = __sinf(x);
  c = __cosf(x);
}

}  // namespace llattn

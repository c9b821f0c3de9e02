// The angle of a rotary position, exact for far ones.
//
// pos x theta is needed modulo a turn.  In turns, theta / 2 pi is a fixed-point
// fraction of 64 bits, F, and pos F modulo 2^64 is an integer product: the error
// of the angle is |pos| 2^-65 turns from F, which is rounded to nearest (2^-41 of a turn at
// 16 million tokens, 2^-32 at 2^33), and 2^-32 of a turn from the final 32 bits.  (In float32 pos x theta itself has
// an error of 0.03 radians at a million tokens; in float64 the products run at a
// sixtieth of the float32 rate.)
#pragma once

#include <stdint.h>

namespace llattn {

// theta / 2 pi as a fraction of 2^64 (modulo 1), to nearest (up to 10^7); theta any finite float32 value.
__device__ __forceinline__ uint64_t rope_turns(float theta) {
  const uint32_t u = __float_as_uint(theta);
  const int e = (int)((u >> 23) & 255);
  const uint64_t m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);  // theta = m 2^-s
  const int s = 150 - (e ? e : 1);
  // hi, lo = m 2 / pi 2^104, from 2 / pi = 0x.a2f9836e4e441529fc2757d1(f534ddc0...): what is cut off is
  // theta 2^-33 of F's last place
  const uint64_t m40 = m << 40, low = m40 * 0xa2f9836e4e441529ull, lo = low + (m * 0xfc2757d1ull << 8);
  const uint64_t hi = __umul64hi(m40, 0xa2f9836e4e441529ull) + (lo < low);
  const int n = s + 42;  // (-62 at least)
  uint64_t f;            // >> n, to nearest
  if (n > 64) f = n < 65 + 64 ? ((hi >> (n - 65)) + 1) >> 1 : 0;  // theta < 2
  else if (n > 0) f = (n < 64 ? hi << (64 - n) | lo >> n : hi) + (lo >> (n - 1) & 1);
  else f = lo << -n;
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

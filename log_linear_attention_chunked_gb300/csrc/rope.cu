// Rotary positions of queries and keys: pairs (a, b) of a head's first `rot`
// elements become amp (a cos - b sin, a sin + b cos), the angle being position x
// inv_freq; backwards (the transpose: gradients) the sine changes sign.
//
// One launch turns queries and keys.  It moves every element once each way and
// bounds on HBM if the angles cost nothing: a thread makes the sines of its pairs
// once and applies them to a group of heads (up to kHeads), 16 bytes of both
// halves of a pair at a time.
#include "la.cuh"
#include "rope.cuh"

namespace llattn {
namespace {

constexpr int kThreads = 256;
// heads that share a thread's sines
constexpr int kHeads = 8;

struct RopeParams {
  int B, H, Hk, T, d, rot, half, groups, units;  // units: of VEC pairs (or copied pieces) in a row
  bool interleaved;
  float amp, sign;
  const float* inv_freq;
  const int64_t* positions;
};

template <typename IO, int N> struct Piece;  // N consecutive elements as float
template <> struct Piece<float, 1> {
  static __device__ __forceinline__ void load(const float* p, float* x) { x[0] = *p; }
  static __device__ __forceinline__ void store(float* p, const float* x) { *p = x[0]; }
};
template <> struct Piece<__nv_bfloat16, 1> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* x) { x[0] = __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) { *p = __float2bfloat16_rn(x[0]); }
};
template <> struct Piece<float, 4> {
  static __device__ __forceinline__ void load(const float* p, float* x) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <> struct Piece<__nv_bfloat16, 8> {
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// VEC elements of each half of VEC pairs to a thread; VEC = 1: of any rot.
template <typename IO, int VEC>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeParams p, const IO* q, const IO* k, IO* qo, IO* ko) {
  const long long at = (long long)(blockIdx.x / p.groups) * kThreads + threadIdx.x;
  const int group = blockIdx.x % p.groups;
  const long long bt = at / p.units;
  if (bt >= (long long)p.B * p.T) return;
  const int u = (int)(at - bt * p.units);
  const int b = (int)(bt / p.T), t = (int)(bt - (long long)b * p.T);
  const int pairs = p.half / VEC;       // units that turn; the others copy
  const bool turn = u < pairs;
  // where the first and the second elements of the pairs stand in a row
  const int i0 = turn ? (p.interleaved ? 2 * u * VEC : u * VEC) : p.rot + (u - pairs) * VEC;
  const int i1 = p.interleaved ? i0 + VEC : i0 + p.half;
  float s[VEC], c[VEC];
  if (turn) {
    const long long pos = p.positions ? p.positions[bt] : t;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      rope_sincos(pos, rope_turns(p.inv_freq[u * VEC + i]), s[i], c[i]);
      s[i] *= p.amp * p.sign;
      c[i] *= p.amp;
    }
  }
  const int h0 = group * kHeads, h1 = min(h0 + kHeads, p.H + p.Hk);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const bool key = h >= p.H;
    const size_t row = key ? ((size_t)b * p.Hk + (h - p.H)) * p.T + t : ((size_t)b * p.H + h) * p.T + t;
    const IO* src = (key ? k : q) + row * p.d;
    IO* dst = (key ? ko : qo) + row * p.d;
    float x[VEC], y[VEC];
    Piece<IO, VEC>::load(src + i0, x);
    if (!turn) {
      Piece<IO, VEC>::store(dst + i0, x);
      continue;
    }
    Piece<IO, VEC>::load(src + i1, y);
    if (VEC > 1 && p.interleaved) {  // pairs lie side by side: (x0 x1) (x2 x3) .. (y0 y1) ..
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        const float a = x[i], bb = x[i + 1], e = y[i], f = y[i + 1];
        x[i] = a * c[i / 2] - bb * s[i / 2];
        x[i + 1] = fmaf(a, s[i / 2], bb * c[i / 2]);
        y[i] = e * c[(VEC + i) / 2] - f * s[(VEC + i) / 2];
        y[i + 1] = fmaf(e, s[(VEC + i) / 2], f * c[(VEC + i) / 2]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float a = x[i], bb = y[i];
        x[i] = a * c[i] - bb * s[i];
        y[i] = fmaf(a, s[i], bb * c[i]);
      }
    }
    Piece<IO, VEC>::store(dst + i0, x);
    Piece<IO, VEC>::store(dst + i1, y);
  }
}

template <typename IO, int VEC> ll_status run(const RopeArgs& a) {
  RopeParams p{a.B, a.H, a.k ? a.Hk : 0, a.T, a.d, a.rope.rot, a.rope.rot / 2, 0, 0, a.rope.interleaved != 0,
               a.rope.amp, a.back ? -1.f : 1.f, a.rope.inv_freq, a.positions};
  p.units = p.half / VEC + (p.d - p.rot) / VEC;
  p.groups = (p.H + p.Hk + kHeads - 1) / kHeads;
  const long long blocks = ((long long)p.B * p.T * p.units + kThreads - 1) / kThreads * p.groups;
  if (blocks > 0x7fffffffll) return LL_ERR_UNSUPPORTED;
  rope_kernel<IO, VEC><<<(unsigned)blocks, kThreads, 0, a.stream>>>(
      p, static_cast<const IO*>(a.q), static_cast<const IO*>(a.k), static_cast<IO*>(a.q_out), static_cast<IO*>(a.k_out));
  LL_CUDA_OK(cudaGetLastError());
  return LL_OK;
}

}  // namespace

// 16 bytes at a time wherever both halves of the pairs (and what is copied) are
// made of whole pieces of 16 bytes; else element by element.
ll_status rope_launch(const RopeArgs& a) {
  const int vec = a.io == LL_F32 ? 4 : 8;
  const bool wide = a.rope.rot / 2 % vec == 0;
  if (a.io == LL_F32) return wide ? run<float, 4>(a) : run<float, 1>(a);
  return wide ? run<__nv_bfloat16, 8>(a) : run<__nv_bfloat16, 1>(a);
}

}  // namespace llattn

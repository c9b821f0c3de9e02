// Rotary positions of queries and keys: pairs (a, b) of a head's first `rot`
// elements become amp (a cos - b sin, a sin + b cos), the angle being position x
// inv_freq; backwards (the transpose: gradients) the sine changes sign.
//
// One launch turns queries and keys.  It moves every element once each way and
// bounds on HBM if the angles cost nothing: a thread makes the sines of its pairs
// once and applies them to a group of heads (up to kHeads), 16 bytes of both
// halves of a pair at a time.  Queries and keys of 2 x 4096 tokens, 32 heads of 128 in all, bf16: 25.2 us a call among
// others (20 at the copy rate); four heads to a thread 28.7, sixteen 26.9 (and single tokens 13.4 where 11.4), CTAs of 256 threads 28.7.
// Captured, behind a flushed L2: 29.8; float32 48; a rotated part of 100, element by element, 77 (float32 82).
#include "la.cuh"
#include "rope.cuh"
#include "sm100.cuh"

namespace llattn {
namespace {

using sm100::pack_bf16x2;

constexpr int kThreads = 128;
// heads that share a thread's sines
constexpr int kHeads = 8;

struct RopeParams {
  int B, H, Hk, T, d, rot, half, groups, units;  // units: of VEC pairs (or copied pieces) in a row
  bool interleaved;
  float amp, sign;
  const float* inv_freq;
  const int64_t* positions;
};

template <typename IO, int N> struct Piece;  // N consecutive elements, as they lie and as float
template <> struct Piece<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ void unpack(Raw v, float* x) { x[0] = v; }
  static __device__ __forceinline__ Raw pack(const float* x) { return x[0]; }
};
template <> struct Piece<__nv_bfloat16, 1> {
  using Raw = __nv_bfloat16;
  static __device__ __forceinline__ void unpack(Raw v, float* x) { x[0] = __bfloat162float(v); }
  static __device__ __forceinline__ Raw pack(const float* x) { return __float2bfloat16_rn(x[0]); }
};
template <> struct Piece<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void unpack(const Raw& v, float* x) {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  static __device__ __forceinline__ Raw pack(const float* x) { return make_float4(x[0], x[1], x[2], x[3]); }
};
template <> struct Piece<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void unpack(const Raw& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Raw pack(const float* x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
};

// VEC elements of each half of VEC pairs to a thread; VEC = 1: of any rot.  The next kBatch heads are on
// their way while these are turned, the first ones while the sines are made.
constexpr int kBatch = 4;
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
  const int i1 = !turn ? i0 : p.interleaved ? i0 + VEC : i0 + p.half;
  const int h0 = group * kHeads, h1 = min(h0 + kHeads, p.H + p.Hk);
  auto row_of = [&](int h) {
    return h >= p.H ? (((size_t)b * p.Hk + (h - p.H)) * p.T + t) * p.d : (((size_t)b * p.H + h) * p.T + t) * p.d;
  };
  using Raw = typename Piece<IO, VEC>::Raw;
  Raw x[kBatch], y[kBatch];
  auto load = [&](int h, Raw& a, Raw& c) {
    const IO* src = (h >= p.H ? k : q) + row_of(h);
    a = *reinterpret_cast<const Raw*>(src + i0);
    c = *reinterpret_cast<const Raw*>(src + i1);
  };
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    if (h0 + j < h1) load(h0 + j, x[j], y[j]);
  float s[VEC], c[VEC];
  if (turn) {
    const long long pos = p.positions ? p.positions[bt] : t;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const uint64_t f = rope_turns(p.inv_freq[u * VEC + i]);
      if (sizeof(IO) == 2) rope_sincos_fast(pos, f, s[i], c[i]);
      else rope_sincos(pos, f, s[i], c[i]);
      s[i] *= p.amp * p.sign;
      c[i] *= p.amp;
    }
  }
#pragma unroll 1
  for (int hb = h0; hb < h1; hb += kBatch) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = hb + j;
      if (h >= h1) break;
      float a[VEC], e[VEC];
      Piece<IO, VEC>::unpack(x[j], a);
      Piece<IO, VEC>::unpack(y[j], e);
      if (h + kBatch < h1) load(h + kBatch, x[j], y[j]);
      IO* dst = (h >= p.H ? ko : qo) + row_of(h);
      if (turn && VEC > 1 && p.interleaved) {  // pairs lie side by side: (a0 a1) (a2 a3) .. (e0 e1) ..
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          const float a0 = a[i], a1 = a[i + 1], e0 = e[i], e1 = e[i + 1];
          a[i] = a0 * c[i / 2] - a1 * s[i / 2];
          a[i + 1] = fmaf(a0, s[i / 2], a1 * c[i / 2]);
          e[i] = e0 * c[(VEC + i) / 2] - e1 * s[(VEC + i) / 2];
          e[i + 1] = fmaf(e0, s[(VEC + i) / 2], e1 * c[(VEC + i) / 2]);
        }
      } else if (turn) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float a0 = a[i], e0 = e[i];
          a[i] = a0 * c[i] - e0 * s[i];
          e[i] = fmaf(a0, s[i], e0 * c[i]);
        }
      }
      *reinterpret_cast<Raw*>(dst + i0) = Piece<IO, VEC>::pack(a);
      if (turn) *reinterpret_cast<Raw*>(dst + i1) = Piece<IO, VEC>::pack(e);
    }
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

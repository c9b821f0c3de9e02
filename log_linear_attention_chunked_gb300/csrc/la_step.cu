// One token of linear attention with a decay per head, for every row of a batch:
//   q, k turned to their position (if asked for),  S <- alpha S + v k^T,  o = scale S q.
//
// Every named state is read and written once, 4 dk dv bytes each way, and that
// bounds it.  A warp takes kRows x (32 / lanes of a row) rows of one state and has
// all of their loads in flight at once, 16 bytes a lane and 512 bytes in a row;
// meanwhile the CTA's threads make the turned key and query, an element each.  The rows'
// sums over the lanes are taken together: each step of the butterfly halves the rows a lane carries.
// Four warps to a CTA and six CTAs to an SM: B 64, 32 heads of 128 x 128, 48 us, 84 % of the measured HBM rate;
// with 85 registers (five CTAs) 61, eight CTAs 50, a CTA to a whole state 52.
#include "la.cuh"
#include "rope.cuh"

namespace llattn {
namespace {

constexpr int kRows = 8;    // 16-byte loads of a lane
constexpr int kWarps = 4;   // at most, of a CTA

struct StepParams {
  int B, H, Hk, dv, parts, n_slots, per_head, rot, interleaved;
  float scale, amp;
  const int64_t* slots;
  const int64_t* positions;
  const float *inv_freq, *log_alpha;
  float* states;
  unsigned* err;
};

__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}

// element i of a head, turned to position `pos`
template <typename IO>
__device__ __forceinline__ float turned(const IO* row, int i, long long pos, const StepParams& p) {
  const float x = to_f(row[i]);
  if (i >= p.rot) return x;
  const int half = p.rot / 2;
  const bool second = p.interleaved ? i & 1 : i >= half;
  const int pair = p.interleaved ? i >> 1 : second ? i - half : i;
  const float y = to_f(row[p.interleaved ? i ^ 1 : second ? i - half : i + half]);
  float s, c;
  rope_sincos(pos, rope_turns(p.inv_freq[pair]), s, c);
  s *= p.amp;
  c *= p.amp;
  return second ? fmaf(y, s, x * c) : x * c - y * s;
}

template <typename IO, int DK>
__global__ void __launch_bounds__(32 * kWarps, 6) la_step_kernel(StepParams p, const IO* q, const IO* k, const IO* v, IO* o) {
  constexpr int LPR = DK / 4, RPI = 32 / LPR;  // lanes of a row, rows of a load
  __shared__ __align__(16) float qk[2 * DK];
  const int lane = threadIdx.x & 31, l = lane % LPR, i0 = 4 * l, warps = blockDim.x >> 5;
  const int part = (int)(blockIdx.x % (unsigned)p.parts);
  const long long bh = blockIdx.x / (unsigned)p.parts;
  const int h = (int)(bh % p.H), b = (int)(bh / p.H);
  const long long slot = p.slots ? p.slots[b] : b;
  if (slot < 0 || slot >= p.n_slots) {  // -1 is a row of padding; anything else out of range an error
    if (slot != -1 && threadIdx.x == 0) raise_error(p.err, kErrDeviceArg);
    return;
  }
  const int r0 = (part * warps + (threadIdx.x >> 5)) * kRows * RPI + lane / LPR;
  float* st = p.states + ((size_t)slot * p.H + h) * p.dv * DK;
  float4 s[kRows];
#pragma unroll
  for (int x = 0; x < kRows; ++x)
    if (r0 + x * RPI < p.dv) s[x] = *reinterpret_cast<const float4*>(st + (size_t)(r0 + x * RPI) * DK + i0);
  float vv[kRows];
#pragma unroll
  for (int x = 0; x < kRows; ++x) vv[x] = r0 + x * RPI < p.dv ? to_f(v[bh * p.dv + r0 + x * RPI]) : 0.f;
  const float la = p.log_alpha[p.per_head ? h : bh];
  const size_t kh = ((size_t)b * p.Hk + h / (p.H / p.Hk)) * DK;
  const long long pos = p.rot ? p.positions[b] : 0;
  for (int e = threadIdx.x; e < 2 * DK; e += blockDim.x) qk[e] = turned((e < DK ? q : k) + kh, e & (DK - 1), pos, p);
  __syncthreads();
  float kx[4], qx[4];
  load4(qk + i0, qx);
  load4(qk + DK + i0, kx);
  // two rows of the batch with one slot would race: one CTA of the row looks
  if (p.slots && part == 0 && h == 0)
    for (int x = threadIdx.x; x < b; x += blockDim.x)
      if (p.slots[x] == slot) raise_error(p.err, kErrDeviceArg);
  const LaDecay d = la_decay(la);
  const bool forget = d.f == 0.f && !d.near;  // whatever the state holds: slots are handed on
  float sum[kRows];
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    sum[x] = 0.f;
    if (r0 + x * RPI < p.dv) {
      float4 y = s[x];
      if (forget) y = make_float4(0.f, 0.f, 0.f, 0.f);
      y.x = fmaf(vv[x], kx[0], la_apply(d, y.x));
      y.y = fmaf(vv[x], kx[1], la_apply(d, y.y));
      y.z = fmaf(vv[x], kx[2], la_apply(d, y.z));
      y.w = fmaf(vv[x], kx[3], la_apply(d, y.w));
      *reinterpret_cast<float4*>(st + (size_t)(r0 + x * RPI) * DK + i0) = y;
      sum[x] = fmaf(y.x, qx[0], y.y * qx[1]) + fmaf(y.z, qx[2], y.w * qx[3]);
    }
  }
  int n = kRows, at = 0;  // rows this lane still carries, and the first of them
  bool writes = true;
#pragma unroll
  for (int w = LPR / 2; w > 0; w >>= 1) {
    const bool up = l & w;
    if (n > 1) {
      n /= 2;
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const float keep = up ? sum[j + n] : sum[j], send = up ? sum[j] : sum[j + n];
        sum[j] = keep + __shfl_xor_sync(0xffffffffu, send, w);
      }
      at += up ? n : 0;
    } else {
      sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], w);
      writes = writes && !up;
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int r = r0 + (at + j) * RPI;
    if (j < n && writes && r < p.dv) o[bh * p.dv + r] = from_f<IO>(p.scale * sum[j]);
  }
}

template <typename IO, int DK> ll_status run(const LaStepArgs& a) {
  constexpr int rows = kRows * 32 / (DK / 4);
  const int warps = (a.dv + rows - 1) / rows;
  const int parts = warps > kWarps ? warps / kWarps : 1;
  StepParams p{a.B, a.H, a.Hk, a.dv, parts, a.n_slots, a.per_head, a.rope.rot, a.rope.interleaved,
               a.scale, a.rope.amp, a.slots, a.positions, a.rope.inv_freq, a.log_alpha, a.states, a.err};
  la_step_kernel<IO, DK><<<(unsigned)((long long)a.B * a.H * parts), 32 * (warps / parts), 0, a.stream>>>(
      p, static_cast<const IO*>(a.q), static_cast<const IO*>(a.k), static_cast<const IO*>(a.v), static_cast<IO*>(a.o));
  LL_CUDA_OK(cudaGetLastError());
  return LL_OK;
}
template <typename IO> ll_status by_dk(const LaStepArgs& a) {
  switch (a.dk) {
    case 16: return run<IO, 16>(a);
    case 32: return run<IO, 32>(a);
    case 64: return run<IO, 64>(a);
    case 128: return run<IO, 128>(a);
  }
  return LL_ERR_UNSUPPORTED;
}

}  // namespace

ll_status la_step_launch(const LaStepArgs& a) {
  return a.io == LL_F32 ? by_dk<float>(a) : by_dk<__nv_bfloat16>(a);
}

}  // namespace llattn

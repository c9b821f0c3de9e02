// Linear attention with a decay per head token by token, states in registers:
// every type and head size, float32 arithmetic throughout.
//
// The forward and all three gradients are the same recurrence over a matrix M
// [rows, columns] with different roles,
//   M_t = a_t M_{t-1} + y_t z_t^T,   out_t = f M_t x_t:
//   o    rows d_v   y = v         z = k    x = q    forwards
//   dq   rows d_k   y = k         z = v    x = do   forwards
//   dk   rows d_k   y = scale q   z = do   x = v    backwards
//   dv   rows d_v   y = scale do  z = q    x = k    backwards
// and a row needs no other row.  A group of kLpr lanes holds kRt rows (kEpl elements
// of each a lane), a CTA a block of rows of one (segment, head).  An element takes
// three operations a token (decay, dot product with the decayed row, update), on
// pairs of floats; what bounds it is reading z and x from shared memory for them (float32, 128 x 128,
// B 2, H 16, T 4096: its pipe 62 to 74 % busy, the operations' 30 to 38; forward 777 us, gradient 1717).  M_t x_t is a M_{t-1} x_t + y_t (z_t . x_t) with the
// scalar products z . x made once per staged tile, which keeps the update out of the
// sum's chain, and gives the part of the sum that lies before token t by itself:
// that is what the decay's gradient is made of,
//   dlog_alpha_t = <S, B> + sum_{j < t} (k_j.dk'_j - q_j.dq'_j),
// over the tokens of the segment, the primes leaving out a token's own pair, S and B the
// state and its gradient at the segment's start, and likewise from the end backwards
// (finish_decay).  (Every partial sum from the start is a dlog_alpha itself; the first ones from a
// sequence's end are taken from a state that no decay has touched yet, and may cancel, which the
// squares of their terms show.)  Sums over the lanes are taken for kLpr
// tokens at once: each step of a butterfly halves the values that a lane carries.
//
// alpha_t is rounded to float32 once a token; what the roundings of a staged tile are off by, those near 1,
// is taken out of the next tile's first, so that those of a constant decay do not add up.
#include <algorithm>

#include "la.cuh"
#include "sm100.cuh"

namespace llattn {
namespace {

using sm100::cp_async16;
using sm100::cp_async_commit;
using sm100::cp_async_wait;

constexpr int kTile = 16;  // tokens staged at a time
constexpr int kMaxThreads = 128;

template <int NC> struct Cfg {
  static constexpr int kEpl = NC >= 64 ? 16 : 8;     // elements of a row in a lane
  static constexpr int kLpr = NC / kEpl;             // lanes per row
  static constexpr int kRt = NC >= 64 ? 2 : 1;       // rows per lane
  static constexpr int kMaxRows = kMaxThreads / kLpr * kRt;
  static constexpr int kPieces = kEpl / 4;
};
// threads and rows of a CTA for `rows` rows in all
template <int NC> int threads_for(int rows) {
  const int t = rows / Cfg<NC>::kRt * Cfg<NC>::kLpr;
  return std::min(kMaxThreads, (t + 31) / 32 * 32);
}
template <int NC> int rows_for(int rows) { return threads_for<NC>(rows) / Cfg<NC>::kLpr * Cfg<NC>::kRt; }
int row_blocks(int rows, int cols) {
  const int r = cols == 128 ? rows_for<128>(rows) : cols == 64 ? rows_for<64>(rows) : cols == 32 ? rows_for<32>(rows)
                                                                                             : rows_for<16>(rows);
  return (rows + r - 1) / r;
}

// ---- pairs of floats
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(f2 a) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
  return make_float2(x, y);
}

struct RecJob {
  const void *y, *z, *x, *w;  // w: rows of the scalar products behind `part`, or null
  bool y_key, z_key, x_key;   // of key heads ([B,Hk,T,..]), else of value heads
  bool rev, trans;            // backwards; rows are d_k (states lie [d_v][d_k])
  int rows;
  float y_scale, f;
  const float* in;            // states on entry, by slot or by sequence; null: zero
  bool in_by_slot;
  void* out;                  // [.., rows] of value heads, io type or float
  bool out_f32;
  float* part;                // [row block][B H T]: w . (a M_{t-1} x_t) f
  float* sum;                 // [slot, H]: the state behind the segment (no outputs)
  float* last;                // [sequence, H]: the state behind the sequence, or null
};
constexpr int kMaxJobs = 3;
struct RecParams {
  GdrSeqs seqs;
  int seg, per_head, dk, dv;
  size_t part_stride;  // B H T
  const float* log_alpha;
  float* log_decay;    // [slot, H], written by the job that sums forwards, or null
  unsigned* err;
  RecJob job[kMaxJobs];
};

template <typename IO> struct Load4;
template <> struct Load4<float> {
  static __device__ __forceinline__ void pairs(const float* p, f2* x) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    x[0] = v.x;
    x[1] = v.y;
  }
};
template <> struct Load4<__nv_bfloat16> {
  static __device__ __forceinline__ void pairs(const __nv_bfloat16* p, f2* x) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = pair(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    x[1] = pair(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
};

template <typename IO, int NC> struct RecSm {
  IO z[2][kTile][NC];
  IO x[2][kTile][NC];
  IO y[2][kTile][Cfg<NC>::kMaxRows];
  IO w[2][kTile][Cfg<NC>::kMaxRows];
  float out[kTile][Cfg<NC>::kMaxRows];
  float red[kTile][4];
  float alpha[2][kTile], zx[kTile];
};

template <typename IO, int NC, bool OUT>
__global__ void __launch_bounds__(kMaxThreads) la_rec_kernel(const __grid_constant__ RecParams p) {
  using C = Cfg<NC>;
  constexpr int LPR = C::kLpr, EPL = C::kEpl, RT = C::kRt;
  __shared__ __align__(16) RecSm<IO, NC> sm;
  la_chain();
  const RecJob& job = p.job[blockIdx.y];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int l = tid % LPR, g = tid / LPR, groups = threads / LPR, cta_rows = groups * RT;
  const int blocks = (job.rows + cta_rows - 1) / cta_rows;
  if ((int)blockIdx.x == 0 && blockIdx.y == 0 && p.seqs.starts)  // every sequence's bounds, whoever finds it
    for (int i = tid; i < p.seqs.n; i += threads) {
      GdrSeq q;
      if (!gdr_seq(p.seqs, i, q)) raise_error(p.err, kErrDeviceArg);
    }
  const long long unit = blockIdx.x / (unsigned)blocks;
  const int rb = (int)(blockIdx.x - unit * blocks), r0 = rb * cta_rows;
  const int h = (int)(unit % p.seqs.H), slot = (int)(unit / p.seqs.H), hk = h / (p.seqs.H / p.seqs.Hk);
  if (rb >= blocks) return;
  LaSegment s;
  if (!la_find(p.seqs, slot, p.seg, s, p.err)) return;
  const int elems = p.dk * p.dv;
  const size_t row = ((size_t)s.row_b * p.seqs.H + h) * p.seqs.T + s.start;
  const size_t krow = ((size_t)s.row_b * p.seqs.Hk + hk) * p.seqs.T + s.start;
  const IO* z = static_cast<const IO*>(job.z) + (job.z_key ? krow : row) * NC;
  const IO* x = static_cast<const IO*>(job.x) + (job.x_key ? krow : row) * NC;
  const IO* y = static_cast<const IO*>(job.y) + (job.y_key ? krow : row) * job.rows + r0;
  const IO* w = OUT && job.w ? static_cast<const IO*>(job.w) + krow * job.rows + r0 : nullptr;
  const float* la = p.log_alpha + (p.per_head ? (size_t)h : row);

  // the state on entry
  f2 m[RT][EPL / 2];
  const float* in = job.in ? job.in + ((size_t)(job.in_by_slot ? slot : s.seq) * p.seqs.H + h) * elems : nullptr;
  auto at = [&](int r, int c) { return job.trans ? (size_t)c * p.dk + r : (size_t)r * p.dk + c; };
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = r0 + i * groups + g;
#pragma unroll
    for (int e = 0; e < EPL / 2; ++e) {
      const int c = ((e >> 1) * LPR + l) * 4 + 2 * (e & 1);
      m[i][e] = in && r < job.rows ? pair(in[at(r, c)], in[at(r, c + 1)]) : 0ull;
    }
  }

  auto token = [&](int i) { return job.rev ? s.n - 1 - i : i; };
  auto stage = [&](int tile) {
    const int b = tile & 1, n = min(kTile, s.n - tile * kTile);
    constexpr int PC = NC * (int)sizeof(IO) / 16;
    for (int e = tid; e < n * PC; e += threads) {
      const int u = e / PC, c = e % PC;
      const size_t o = (size_t)token(tile * kTile + u) * NC;
      cp_async16(reinterpret_cast<char*>(sm.z[b][u]) + 16 * c, reinterpret_cast<const char*>(z + o) + 16 * c);
      if (OUT) cp_async16(reinterpret_cast<char*>(sm.x[b][u]) + 16 * c, reinterpret_cast<const char*>(x + o) + 16 * c);
    }
    const int pr = min(cta_rows, job.rows - r0) * (int)sizeof(IO) / 16;
    for (int e = tid; e < n * pr; e += threads) {
      const int u = e / pr, c = e % pr;
      const size_t o = (size_t)token(tile * kTile + u) * job.rows;
      cp_async16(reinterpret_cast<char*>(sm.y[b][u]) + 16 * c, reinterpret_cast<const char*>(y + o) + 16 * c);
      if (OUT && w) cp_async16(reinterpret_cast<char*>(sm.w[b][u]) + 16 * c, reinterpret_cast<const char*>(w + o) + 16 * c);
    }
    cp_async_commit();
  };
  // the log decay that M is multiplied by before its i-th token: backwards that of the
  // token just done (what comes in is already decayed to the segment's border)
  auto log_alpha = [&](int i) {
    if (i >= s.n || (job.rev && i == 0)) return 0.f;
    return la_log(la[p.per_head ? 0 : job.rev ? s.n - i : i]);
  };
  const int tiles = (s.n + kTile - 1) / kTile;
  float g_next = 0.f, off = 0.f;
  double g_all = 0.;
  if (tiles > 0) {
    stage(0);
    if (warp == 0 && lane < kTile) g_next = log_alpha(lane);
  }
  for (int tile = 0; tile < tiles; ++tile) {
    const int b = tile & 1, n = min(kTile, s.n - tile * kTile);
    cp_async_wait<0>();
    if (warp == 0) {  // this tile's decays
      const float ga = g_next;
      if (lane < kTile) g_next = log_alpha((tile + 1) * kTile + lane);
      g_all += lane < kTile ? (double)ga : 0.;
      const bool near = ga > -0.5f && lane < kTile;
      float a = near ? expm1f(ga) : expf(ga), left = 0.f;
      if (near) {
        const float d = lane == 0 ? a - off : a;
        a = 1.f + d;
        left = (a - 1.f) - d;
      }
      off = __shfl_sync(0xffffffffu, near ? 0.f : off, 0);  // (a first token that is not near leaves it to the next tile)
#pragma unroll
      for (int o = kTile / 2; o > 0; o >>= 1) left += __shfl_xor_sync(0xffffffffu, left, o);
      off += __shfl_sync(0xffffffffu, left, 0);
      if (lane < kTile) sm.alpha[b][lane] = a;
    }
    __syncthreads();
    if (tile + 1 < tiles) stage(tile + 1);
    if (OUT) {  // z . x, a token to LPR lanes
      for (int u = g; u < kTile; u += groups) {
        float t = 0.f;
        if (u < n) {
          f2 acc = 0ull;
#pragma unroll
          for (int c = 0; c < C::kPieces; ++c) {
            f2 zz[2], xx[2];
            Load4<IO>::pairs(&sm.z[b][u][(c * LPR + l) * 4], zz);
            Load4<IO>::pairs(&sm.x[b][u][(c * LPR + l) * 4], xx);
            acc = fma2(zz[0], xx[0], acc);
            acc = fma2(zz[1], xx[1], acc);
          }
          const float2 v = unpair(acc);
          t = v.x + v.y;
        }
        // (groups divides kTile or is a multiple of it: whole groups come here, and LPR lanes of a warp together)
        const uint32_t mask = (LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << (lane / LPR * LPR));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) t += __shfl_xor_sync(mask, t, o);
        if (l == 0) sm.zx[u] = t;
      }
      __syncthreads();
    }
#pragma unroll 1
    for (int u0 = 0; u0 < kTile; u0 += LPR) {
      if (u0 >= n) break;
      float pre[RT][LPR];
#pragma unroll
      for (int u = 0; u < LPR; ++u) {
        if (u0 + u >= n) {
#pragma unroll
          for (int i = 0; i < RT; ++i) pre[i][u] = 0.f;
          continue;
        }
        const float a = sm.alpha[b][u0 + u];
        const f2 aa = pair(a, a);
        f2 yy[RT], acc[RT][2];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float yv = to_f(sm.y[b][u0 + u][i * groups + g]) * job.y_scale;
          yy[i] = pair(yv, yv);
          acc[i][0] = acc[i][1] = 0ull;
        }
#pragma unroll
        for (int c = 0; c < C::kPieces; ++c) {
          f2 zz[2], xx[2];
          Load4<IO>::pairs(&sm.z[b][u0 + u][(c * LPR + l) * 4], zz);
          if (OUT) Load4<IO>::pairs(&sm.x[b][u0 + u][(c * LPR + l) * 4], xx);
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const f2 d = mul2(m[i][2 * c + e], aa);
              if (OUT) acc[i][e] = fma2(d, xx[e], acc[i][e]);
              m[i][2 * c + e] = fma2(yy[i], zz[e], d);
            }
        }
        if (OUT)
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float2 v0 = unpair(acc[i][0]), v1 = unpair(acc[i][1]);
            pre[i][u] = (v0.x + v0.y) + (v1.x + v1.y);
          }
      }
      if (OUT) {
        // lane l of a group ends with the sum of token u0 + l
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          int cnt = LPR;
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) {
            const bool up = l & o;
            cnt /= 2;
#pragma unroll
            for (int j = 0; j < LPR / 2; ++j)
              if (j < cnt) {
                const float keep = up ? pre[i][j + cnt] : pre[i][j], send = up ? pre[i][j] : pre[i][j + cnt];
                pre[i][j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
              }
          }
          const int u = u0 + l, rr = i * groups + g;
          if (u < n && r0 + rr < job.rows) {
            const float own = to_f(sm.y[b][u][rr]) * job.y_scale * sm.zx[u];
            sm.out[u][rr] = job.f * (pre[i][0] + own);
            if (w) dot = fmaf(to_f(sm.w[b][u][rr]), pre[i][0], dot);
          }
        }
        if (w) {
#pragma unroll
          for (int o = LPR; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
          if (lane < LPR && u0 + lane < kTile) sm.red[u0 + lane][warp] = dot;
        }
      }
    }
    if (OUT) {
      __syncthreads();
      const int nr = min(cta_rows, job.rows - r0);
      for (int e = tid; e < n * nr; e += threads) {
        const int u = e / nr, rr = e % nr;
        const size_t o = (row + token(tile * kTile + u)) * job.rows + r0 + rr;
        if (job.out_f32) static_cast<float*>(job.out)[o] = sm.out[u][rr];
        else static_cast<IO*>(job.out)[o] = from_f<IO>(sm.out[u][rr]);
      }
      if (w && tid < n) {
        float t = 0.f;
        for (int k = 0; k < threads / 32; ++k) t += sm.red[tid][k];
        job.part[rb * p.part_stride + row + token(tile * kTile + tid)] = job.f * t;
      }
    }
  }

  // what leaves the segment (backwards: at the border before its first token)
  float* dst = !OUT ? job.sum + ((size_t)slot * p.seqs.H + h) * elems
               : job.last && (job.rev ? s.num == 0 : (long long)s.num * p.seg + s.n == s.seq_len)
                   ? job.last + ((size_t)s.seq * p.seqs.H + h) * elems : nullptr;
  if (dst) {
    const LaDecay d = job.rev && s.n > 0 ? la_decay(la_log(la[0])) : LaDecay{0.f, true};
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = r0 + i * groups + g;
      if (r < job.rows)
#pragma unroll
        for (int e = 0; e < EPL / 2; ++e) {
          const int c = ((e >> 1) * LPR + l) * 4 + 2 * (e & 1);
          const float2 v = unpair(m[i][e]);
          dst[at(r, c)] = la_apply(d, v.x);
          dst[at(r, c + 1)] = la_apply(d, v.y);
        }
    }
  }
  if (!OUT && !job.rev && rb == 0 && warp == 0 && p.log_decay) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) g_all += __shfl_xor_sync(0xffffffffu, g_all, o);
    if (lane == 0) p.log_decay[(size_t)slot * p.seqs.H + h] = (float)g_all;
  }
}

// ---------------------------------------------------------------- along the segments
// Four elements to a thread, some CTAs to a (sequence, head).  The loads of four
// segments travel together.
constexpr int kCarryThreads = 128;
__global__ void __launch_bounds__(kCarryThreads) la_carry_kernel(LaCarry c) {
  la_chain();
  const int dir = blockIdx.y;
  float* sums = c.sums[dir];
  if (!sums) return;
  const int per = (c.elems / 4 + kCarryThreads - 1) / kCarryThreads, row = blockIdx.x / per;
  const int h = row % c.seqs.H, seq = row / c.seqs.H;
  const int e = ((int)(blockIdx.x - (unsigned)row * per) * kCarryThreads + threadIdx.x) * 4;
  if (e >= c.elems) return;
  GdrSeq q;
  if (!gdr_seq(c.seqs, seq, q)) return;
  const int base = gdr_slot_base(c.seqs, seq, q.start, c.seg), n = (q.len + c.seg - 1) / c.seg;
  const size_t sh = (size_t)seq * c.seqs.H + h;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c.init[dir]) x = *reinterpret_cast<const float4*>(c.init[dir] + sh * c.elems + e);
  if (n == 0) *reinterpret_cast<float4*>(sums + ((size_t)base * c.seqs.H + h) * c.elems + e) = x;  // (an empty sequence's slot)
  for (int i0 = 0; i0 < n; i0 += 4) {
    float4 y[4];
    LaDecay d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j < n - 1) {  // (nothing needs the last one's sum)
        const size_t at = (size_t)(base + (dir ? n - 1 - i0 - j : i0 + j)) * c.seqs.H + h;
        y[j] = *reinterpret_cast<const float4*>(sums + at * c.elems + e);
        d[j] = la_decay(c.log_decay[at]);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j < n) {
        const size_t at = (size_t)(base + (dir ? n - 1 - i0 - j : i0 + j)) * c.seqs.H + h;
        *reinterpret_cast<float4*>(sums + at * c.elems + e) = x;
        if (i0 + j == n - 1) break;
        x.x = la_apply(d[j], x.x) + y[j].x;
        x.y = la_apply(d[j], x.y) + y[j].y;
        x.z = la_apply(d[j], x.z) + y[j].z;
        x.w = la_apply(d[j], x.w) + y[j].w;
      }
  }
}

// ---------------------------------------------------------------- the decay's gradient, shared heads
struct FinishParams {
  GdrSeqs seqs;
  int seg, dk, dv, per_head, parts;
  size_t part_stride;
  const float *log_alpha, *part_q, *part_k;  // [row block][B H T]
  const float* entry;                        // states on entry, by slot or by sequence; null: zero
  bool by_slot;
  const float* behind;                       // gradients at the segments' ends by slot,
  const float* first;                        // before the sequences
  float* copy_first;                         // where `first` goes, or null
  const float *after, *dstate_out;           // behind the sequences: states and their gradients, or null
  float* dlog_alpha;
  double* head_sums;                         // [slot, H] when log_alpha is one to a head
  const float *dq, *dkey;                    // [B,H,T,dk] float32, shared heads
  void *dq_out, *dk_out;
  unsigned segments, key_rows;               // CTAs of the decays; B Hk T of shared heads
};
constexpr int kFinishThreads = 512;
constexpr int kFinishKept = 3;  // every segment in chunks (at most 12 of 128 tokens)
__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float2 pair_sum(float2 x) {  // over a warp
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x = pair_add(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o)));
  return x;
}
// dq and dk of a key head: its value heads' in their order, four elements to a thread (key_rows below 2^30)
template <typename IO> __device__ __forceinline__ void store4(IO* d, float4 x);
template <> __device__ __forceinline__ void store4<float>(float* d, float4 x) { *reinterpret_cast<float4*>(d) = x; }
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* d, float4 x) {
  *reinterpret_cast<uint2*>(d) = make_uint2(sm100::pack_bf16x2(x.x, x.y), sm100::pack_bf16x2(x.z, x.w));
}
template <typename IO> __device__ __forceinline__ void sum_heads(const FinishParams& p, unsigned block) {
  const unsigned n4 = p.dk / 4, per = kFinishThreads / n4, G = p.seqs.H / p.seqs.Hk, T = p.seqs.T;  // rows of a CTA
  const unsigned krow = (block >> 1) * per + threadIdx.x / n4, c = threadIdx.x % n4;
  if (krow >= p.key_rows) return;
  const unsigned bk = krow / T, t = krow - bk * T;
  if (p.seqs.starts && ((int)t < p.seqs.starts[0] || (int)t >= p.seqs.starts[p.seqs.n])) return;  // of no sequence
  const float4* a = reinterpret_cast<const float4*>((block & 1 ? p.dkey : p.dq) + ((size_t)bk * G * T + t) * p.dk) + c;
  const size_t head = (size_t)T * n4;
  float4 x = *a;
#pragma unroll 4
  for (unsigned i = 1; i < G; ++i) {
    const float4 y = a[i * head];
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  }
  store4(static_cast<IO*>(block & 1 ? p.dk_out : p.dq_out) + (size_t)krow * p.dk + 4 * c, x);
}
// The decay's gradient of one (segment, head).  It is a running sum whose values at both ends of the segment, and at
// tokens that forget (zero), are known, so that each token has two values, one summed up from the left and one from
// the right, and each is off by the roundings of the terms that it went over.  Taken alone, the left one hands those of
// large early terms to every later token, however short the memory has become (1e-2 of a token's own terms
// behind values 256 times as large).  The two are joined by the squares of the terms on either side, as independent
// errors ask for: what the sums differ by goes to where the large terms are.  Sums are pairs of
// floats (in float64, two operations a cycle and SM, they took 40 of 52 us for 320 segments).
struct Side {  // a sum towards one side, and of squares; `cut`: it begins at a known value
  float2 s;
  float w;
  bool cut;
};
__device__ __forceinline__ Side join(const Side& near, const Side& far) {  // of what is nearer and what lies behind it
  return near.cut ? near : Side{pair_add(far.s, near.s), far.w + near.w, far.cut};
}
__device__ __forceinline__ Side side_of(const Side& x, int lane) {
  return Side{make_float2(__shfl_sync(0xffffffffu, x.s.x, lane), __shfl_sync(0xffffffffu, x.s.y, lane)),
              __shfl_sync(0xffffffffu, x.w, lane), __shfl_sync(0xffffffffu, (int)x.cut, lane) != 0};
}
// everything up to this lane, from the left (dir = -1) or the right (1)
__device__ __forceinline__ Side scan_side(Side x, int lane, int dir) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int from = lane + dir * o;
    const Side y = side_of(x, from & 31);
    if (from >= 0 && from < 32) x = join(x, y);
  }
  return x;
}
// k.dk (v.dv) and q.dq of a token, and what the sum changes by behind it
struct Term {
  float2 x;
  float k, q;
};
constexpr int kMostParts = 4;  // row blocks of 128 rows (row_blocks), halves of the columns in chunks
static_assert(std::min({Cfg<16>::kMaxRows, Cfg<32>::kMaxRows, Cfg<64>::kMaxRows, Cfg<128>::kMaxRows}) * kMostParts >= 128, "");
__device__ __forceinline__ Term finish_term(const FinishParams& p, size_t at) {
  float k[kMostParts], q[kMostParts];
#pragma unroll
  for (int i = 0; i < kMostParts; ++i)
    if (i < p.parts) {
      k[i] = p.part_k[i * p.part_stride + at];
      q[i] = p.part_q[i * p.part_stride + at];
    }
  Term y{make_float2(0.f, 0.f), 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kMostParts; ++i)
    if (i < p.parts) {
      y.x = pair_add(y.x, make_float2(k[i], 0.f));
      y.x = pair_add(y.x, make_float2(-q[i], 0.f));
      y.k += k[i];
      y.q += q[i];
    }
  return y;
}
// KEPT: tokens of a thread that stay in registers (in segments of up to KEPT x kFinishThreads), 0: read again for each pass
template <int KEPT> __device__ __forceinline__ void finish_decay(const FinishParams& p, const LaSegment& s, int slot, int h) {
  constexpr int W = kFinishThreads / 32;
  static_assert(W <= 32, "a lane to each warp's sum");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t row = ((size_t)s.row_b * p.seqs.H + h) * p.seqs.T + s.start;
  __shared__ float2 red[2][W];
  __shared__ float most[W];
  __shared__ Side warps[2][W];
  const int elems = p.dk * p.dv;
  // <S, B> at the segment's start and at its end
  const bool last = (long long)s.num * p.seg + s.n == s.seq_len;
  auto at = [&](const float* x, int i) { return x ? reinterpret_cast<const float4*>(x + ((size_t)i * p.seqs.H + h) * elems) : nullptr; };
  const float4* B = s.num > 0 ? at(p.behind, slot - 1) : at(p.first, s.seq);
  const float4* S = B ? at(p.entry, p.by_slot ? slot : s.seq) : nullptr;
  const float4* S1 = last ? at(p.after, s.seq) : at(p.entry, slot + 1);
  const float4* B1 = p.by_slot ? at(p.behind, slot) : at(p.dstate_out, s.seq);
  float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int e = tid; e < elems / 4; e += kFinishThreads) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 x = S ? S[e] : z, y = S ? B[e] : z, x1 = S1 ? S1[e] : z, y1 = S1 ? B1[e] : z;
    d0[0] = fmaf(x.x, y.x, d0[0]);
    d0[1] = fmaf(x.y, y.y, d0[1]);
    d0[2] = fmaf(x.z, y.z, d0[2]);
    d0[3] = fmaf(x.w, y.w, d0[3]);
    d1[0] = fmaf(x1.x, y1.x, d1[0]);
    d1[1] = fmaf(x1.y, y1.y, d1[1]);
    d1[2] = fmaf(x1.z, y1.z, d1[2]);
    d1[3] = fmaf(x1.w, y1.w, d1[3]);
  }
  const float2 border = pair_sum(pair_add(pair_add(make_float2(d0[0], 0.f), make_float2(d0[1], 0.f)),
                                          pair_add(make_float2(d0[2], 0.f), make_float2(d0[3], 0.f))));
  const float2 end = pair_sum(pair_add(pair_add(make_float2(d1[0], 0.f), make_float2(d1[1], 0.f)),
                                       pair_add(make_float2(d1[2], 0.f), make_float2(d1[3], 0.f))));
  const int run = (s.n + kFinishThreads - 1) / kFinishThreads, t0 = min(tid * run, s.n), t1 = min(t0 + run, s.n);
  auto forgets = [&](int t) { return gdr_forgets(p.log_alpha[p.per_head ? (size_t)h : row + t]); };
  Term kept[KEPT > 0 ? KEPT : 1];
  bool cuts[KEPT > 0 ? KEPT : 1];
#pragma unroll
  for (int j = 0; j < KEPT; ++j)
    if (t0 + j < t1) {
      kept[j] = finish_term(p, row + t0 + j);
      cuts[j] = forgets(t0 + j);
    }
  auto term = [&](int j) { return KEPT > 0 ? kept[j] : finish_term(p, row + t0 + j); };
  auto cut_at = [&](int j) { return KEPT > 0 ? cuts[j] : forgets(t0 + j); };
  const int most_run = KEPT > 0 ? KEPT : run, own = t1 - t0;
  // the largest term, which the squares are of a part of
  float most_mine = 0.f;
#pragma unroll
  for (int j = 0; j < most_run; ++j)
    if (j < own) {
      const Term y = term(j);
      most_mine = fmaxf(most_mine, fmaxf(fabsf(y.k), fabsf(y.q)));
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most_mine = fmaxf(most_mine, __shfl_xor_sync(0xffffffffu, most_mine, o));
  if (lane == 0) {
    red[0][warp] = border;
    red[1][warp] = end;
    most[warp] = most_mine;
  }
  __syncthreads();
  if (p.copy_first && s.num == 0)  // (this CTA alone reads what stands there, and has)
    for (int e = tid; e < elems / 4; e += kFinishThreads)
      reinterpret_cast<float4*>(p.copy_first + ((size_t)s.seq * p.seqs.H + h) * elems)[e] = B[e];
  const float2 z = make_float2(0.f, 0.f);
  const float2 start_at = pair_sum(lane < W ? red[0][lane % W] : z), end_at = pair_sum(lane < W ? red[1][lane % W] : z);
  float top = lane < W ? most[lane % W] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float unit = top >= 1e-37f ? 1.f / top : 0.f;

  auto square = [&](const Term& y) {
    const float k = y.k * unit, q = y.q * unit;
    return fmaf(k, k, q * q);
  };
  auto minus = [](float2 x) { return make_float2(-x.x, -x.y); };
  const Side none{z, 0.f, false};
  Side l = none, r = none;  // over this thread's tokens
#pragma unroll
  for (int j = 0; j < most_run; ++j)
    if (j < own) {
      const Term y = term(j);
      const float w = square(y);
      if (cut_at(j)) {
        l = Side{z, 0.f, true};
        r.cut = true;
      }
      l.s = pair_add(l.s, y.x);
      l.w += w;
      if (!r.cut) {
        r.s = pair_add(r.s, minus(y.x));
        r.w += w;
      }
    }
  l = scan_side(l, lane, -1);
  r = scan_side(r, lane, 1);
  if (lane == 31) warps[0][warp] = l;
  if (lane == 0) warps[1][warp] = r;
  l = side_of(l, (lane - 1) & 31);
  r = side_of(r, (lane + 1) & 31);
  if (lane == 0) l = none;
  if (lane == 31) r = none;
  __syncthreads();
  Side lw = scan_side(lane < W ? warps[0][lane % W] : none, lane, -1), rw = scan_side(lane < W ? warps[1][lane % W] : none, lane, 1);
  lw = side_of(lw, (warp - 1) & 31);
  rw = side_of(rw, (warp + 1) & 31);
  if (warp == 0) lw = none;
  if (warp == W - 1) rw = none;
  l = join(l, join(lw, Side{start_at, 0.f, true}));
  r = join(r, join(rw, Side{end_at, 0.f, true}));
  float2 all = z;
  float apart = 0.f, squares = 0.f;  // of this piece: what its two sums differ by; all its squares
#pragma unroll
  for (int j = 0; j < most_run; ++j)
    if (j < own) {
      const bool cut = cut_at(j);
      if (cut) l = Side{z, 0.f, true};
      if (cut || j == 0) {  // as far as the next token that forgets, or on to what comes from the right
        Side y = none;
#pragma unroll
        for (int u = j; u < most_run && (KEPT > 0 || !y.cut); ++u)
          if (u < own && !y.cut) {
            const Term x = term(u);
            if (u > j && cut_at(u)) {
              y.cut = true;
            } else {
              y.s = pair_add(y.s, minus(x.x));
              y.w += square(x);
            }
          }
        y = join(y, r);
        const float2 d = pair_add(y.s, minus(l.s));
        apart = d.x + d.y;
        squares = l.w + y.w;
      }
      const Term x = term(j);
      const float2 y = pair_add(l.s, make_float2(squares == 0.f ? 0.f : apart * (l.w / squares), 0.f));
      const float g = cut ? 0.f : y.x + y.y;
      if (p.per_head) all = pair_add(all, make_float2(g, 0.f));
      else p.dlog_alpha[row + t0 + j] = g;
      l.s = pair_add(l.s, x.x);
      l.w += square(x);
    }
  if (p.per_head) {
    all = pair_sum(all);
    if (lane == 0) red[0][warp] = all;  // (every warp has read it before the barrier above)
    __syncthreads();
    all = pair_sum(lane < W ? red[0][lane % W] : z);
    if (tid == 0) p.head_sums[(size_t)slot * p.seqs.H + h] = (double)all.x + (double)all.y;
  }
}
template <typename IO> __global__ void __launch_bounds__(kFinishThreads) la_finish_kernel(FinishParams p) {
  la_chain();
  if (blockIdx.x >= p.segments) return sum_heads<IO>(p, blockIdx.x - p.segments);
  const int h = blockIdx.x % p.seqs.H, slot = blockIdx.x / p.seqs.H;
  LaSegment s;
  if (!la_find(p.seqs, slot, p.seg, s, nullptr) || s.n == 0) {
    if (p.per_head && threadIdx.x == 0) p.head_sums[(size_t)slot * p.seqs.H + h] = 0.;
  } else if (s.n <= kFinishKept * kFinishThreads) {
    finish_decay<kFinishKept>(p, s, slot, h);
  } else {
    finish_decay<0>(p, s, slot, h);
  }
}
__global__ void __launch_bounds__(128) la_head_sum_kernel(const double* sums, int slots, int H, float* out) {
  la_chain();
  __shared__ double red[4];
  const int h = blockIdx.x;
  double x = 0.;
  for (int i = threadIdx.x; i < slots; i += 128) x += sums[(size_t)i * H + h];
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x == 0) out[h] = (float)(red[0] + red[1] + red[2] + red[3]);
}

// ---------------------------------------------------------------- host
// Tokens of a segment: as many segments as keep about four CTAs on every SM (a
// split costs another pass over keys and values, half of the forward's work),
// none below 64 tokens.
int rec_segment(const LaArgs& a) {
  const int blocks = row_blocks(a.dv, a.dk);
  const long long per = ((long long)a.B * a.T * a.H * blocks + 607) / 608;
  const long long seg = std::max<long long>(64, (per + kTile - 1) / kTile * kTile);
  return (int)std::min<long long>(seg, a.T);
}

template <typename IO, int NC, bool OUT>
ll_status rec_run(const RecParams& p, int jobs, size_t slots, cudaStream_t stream, bool after) {
  const int rows = p.job[0].rows, threads = threads_for<NC>(rows), cta = rows_for<NC>(rows);
  const size_t grid = slots * p.seqs.H * ((rows + cta - 1) / cta);
  if (grid > 0x7fffffffull) return LL_ERR_UNSUPPORTED;
  return la_launch(after, la_rec_kernel<IO, NC, OUT>, dim3((unsigned)grid, jobs), threads, 0, stream, p);
}
// jobs of one launch have the same numbers of rows and columns
template <bool OUT>
ll_status rec_launch(ll_dtype io, int cols, const RecParams& p, int jobs, size_t slots, cudaStream_t st, bool after) {
  const bool f = io == LL_F32;
  switch (cols) {
    case 16:
      return f ? rec_run<float, 16, OUT>(p, jobs, slots, st, after) : rec_run<__nv_bfloat16, 16, OUT>(p, jobs, slots, st, after);
    case 32:
      return f ? rec_run<float, 32, OUT>(p, jobs, slots, st, after) : rec_run<__nv_bfloat16, 32, OUT>(p, jobs, slots, st, after);
    case 64:
      return f ? rec_run<float, 64, OUT>(p, jobs, slots, st, after) : rec_run<__nv_bfloat16, 64, OUT>(p, jobs, slots, st, after);
    case 128:
      return f ? rec_run<float, 128, OUT>(p, jobs, slots, st, after) : rec_run<__nv_bfloat16, 128, OUT>(p, jobs, slots, st, after);
  }
  return LL_ERR_UNSUPPORTED;
}
RecParams rec_params(const LaArgs& a, int seg) {
  RecParams p{};
  p.seqs = la_seqs(a);
  p.seg = seg;
  p.per_head = a.per_head;
  p.dk = a.dk;
  p.dv = a.dv;
  p.part_stride = (size_t)a.B * a.H * a.T;
  p.log_alpha = a.log_alpha;
  p.err = a.err;
  return p;
}
RecJob job_o(const LaArgs& a) {
  RecJob j{};
  j.y = a.v;
  j.z = a.k;
  j.x = a.q;
  j.z_key = j.x_key = true;
  j.rows = a.dv;
  j.y_scale = 1.f;
  j.f = a.scale;
  return j;
}
RecJob job_dv(const LaArgs& a) {
  RecJob j{};
  j.y = a.dout;
  j.z = a.q;
  j.x = a.k;
  j.z_key = j.x_key = true;
  j.rev = true;
  j.rows = a.dv;
  j.y_scale = a.scale;
  j.f = 1.f;
  return j;
}
size_t elems_of(const LaArgs& a) { return (size_t)a.dk * a.dv; }

ll_status carry_launch(const LaCarry& c, int sequences, cudaStream_t stream) {
  const size_t grid = (size_t)sequences * c.seqs.H * ((c.elems / 4 + kCarryThreads - 1) / kCarryThreads);
  if (grid > 0x7fffffffull) return LL_ERR_UNSUPPORTED;
  return la_launch(true, la_carry_kernel, dim3((unsigned)grid, c.sums[1] ? 2 : 1), kCarryThreads, 0, stream, c);
}

// ---- in chunks: tokens of a segment, a multiple of a chunk.  More segments fill more
// SMs, and each costs the states' way between them and the filling of its pipeline.  The
// times are those measured at d = 128, in us: a chunk 3.1, of the gradient's jobs 7, of the sums 1.4 (1.9),
// a segment's beginning and end 9, 12, 6.  With smaller heads all of them shrink alike: at 64 and mixed sizes what
// is chosen took at most 7 % more than the best of one to 32 chunks (1 x 8 heads of 8192 tokens, d 64, gradient: 114 us
// where 107), at 128 2 %.  Of packed sequences only the device knows the lengths: their
// work is taken as spread evenly, with half a segment at the end of it.  (Gradient, B 2, H 16, T 4096, segments of
// 6, 8, 11, 12 chunks: 241, 241, 218, 231 us; 7 packed sequences of 5003 tokens, 3, 6, 8, 11: 281, 226, 220, 362.)
// The decay's gradient is summed over a segment, and its rounding with it: at most 12 chunks there.
constexpr int kChunk = 128, kMostGradChunks = 12;
int tc_segment(const LaArgs& a, bool bwd) {
  const double chunk_us = bwd ? 7. : 3.1, fill_us = bwd ? 12. : 9., sum_us = bwd ? 1.9 : 1.4, sum_fill_us = 6.;
  const long long chunks = ((long long)a.T + kChunk - 1) / kChunk;
  const int jobs = bwd ? 3 : 1, dirs = bwd ? 2 : 1, sms = 152;
  double best = 1e30;
  long long seg = chunks;
  for (long long n = 1; n <= chunks && n <= 2 * sms; ++n) {
    const long long per = n == 2 * sms ? std::min<long long>((chunks + n - 1) / n, kMostGradChunks) : (chunks + n - 1) / n;
    if (bwd && per > kMostGradChunks) continue;
    double t;
    if (a.n_seqs) {
      const double slots = ((double)chunks / per + a.n_seqs) * a.H, work = (chunks + 0.5 * a.n_seqs) * a.H;
      t = jobs * (slots * fill_us + work * chunk_us) / sms + std::max(0.5 * per * chunk_us, 1. * fill_us);
      if (n > 1) t += dirs * (slots * sum_fill_us + work * sum_us) / sms + 0.5 * per * sum_us + 6.;
    } else {
      const double slots = (double)a.B * ((chunks + per - 1) / per) * a.H;
      t = std::ceil(slots * jobs / sms) * (per * chunk_us + fill_us);
      if (n > 1) t += std::ceil(slots * dirs / sms) * (per * sum_us + sum_fill_us) + 5. + 0.1 * n;
    }
    if (t < best) {
      best = t;
      seg = per;
    }
  }
  if (bwd) seg = std::min<long long>(seg, kMostGradChunks);
  return (int)std::min<long long>(seg * kChunk, 1ll << 30);
}
// Which of the two ways is the faster (token by token / in chunks, us of a captured call with states behind a flushed L2; mean
// lengths of 16, 32, 64 tokens):
//   128 x 128, 4 heads      forward 13/22, 18/22, 26/22       gradient 24/36, 28/34, 36/34
//              256 heads    forward 30/38, 44/39, 71/40       gradient 83/99, 120/97, 198/99
//              2048 heads   forward 170/221, 259/224, 452/231 gradient 596/659, 861/649, 1443/651
//   64 x 64,   32 heads     forward 14/15, 21/14, 29/15       gradient 23/31, 27/31, 37/31
//              256 heads    forward 16/25, 23/25, 35/26       gradient 37/76, 51/76, 80/76
//              2048 heads   forward 55/132, 85/133, 143/133   gradient 199/480, 284/478, 454/479
//   64 x 128,  4 heads      forward 15/17, 20/17, 30/17       gradient 40/28, 47/30, 71/30
//              256 heads    forward 22/29, 31/29, 47/29       gradient 56/84, 80/83, 125/83
//              2048 heads   forward 100/160, 154/160, 263/162 gradient 340/549, 490/541, 795/542
// (128 x 64 as 64 x 128: 2048 heads forward 90/167, 137/169, 234/171.  Token by token their gradient takes a launch more.)
bool tc_use(const LaArgs& a, bool bwd) {
  if (!la_tc_formats(a)) return false;
  const int mean = a.n_seqs ? (a.T + a.n_seqs - 1) / a.n_seqs : a.T;
  const bool few = (long long)la_sequences(a) * a.H <= 152;
  if (a.dk != a.dv) return mean >= (few ? (bwd ? 8 : 24) : 40);
  if (a.dk == 128) return mean >= (few ? 48 : 24);
  return mean >= (few ? 16 : 48) + (bwd ? 16 : 0);
}

struct Plan {
  bool tc, split;  // in chunks; more than one segment
  int seg, parts;
  size_t slots, sum_s, sum_a, first, after, dec, part_q, part_k, dq, dk, heads, total;
};
// (the workspace cannot depend on which optional tensors a call brings)
Plan plan_of(const LaArgs& a, bool bwd) {
  Plan pl{};
  pl.tc = tc_use(a, bwd);
  pl.seg = pl.tc ? tc_segment(a, bwd) : rec_segment(a);
  pl.slots = la_slots(a, pl.seg);
  pl.split = la_split(a, pl.seg);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align_up(bytes, 256);
    return o;
  };
  const size_t states = pl.slots * a.H * elems_of(a) * 4, tokens = (size_t)a.B * a.H * a.T;
  if (pl.split) {
    pl.sum_s = take(states);
    pl.dec = take(pl.slots * a.H * 4);
  }
  if (bwd) {
    pl.parts = pl.tc ? 2 : row_blocks(a.dk, a.dv);
    if (pl.split) pl.sum_a = take(states);
    pl.first = take((size_t)la_sequences(a) * a.H * elems_of(a) * 4);
    pl.after = take((size_t)la_sequences(a) * a.H * elems_of(a) * 4);
    pl.part_q = take(tokens * pl.parts * 4);
    pl.part_k = take(tokens * pl.parts * 4);
    if (a.H != a.Hk) {
      pl.dq = take(tokens * a.dk * 4);
      pl.dk = take(tokens * a.dk * 4);
    }
    if (a.per_head) pl.heads = take(pl.slots * a.H * 8);
  }
  pl.total = at;
  return pl;
}

}  // namespace

size_t la_fwd_workspace(const LaArgs& a) { return plan_of(a, false).total; }
int la_fwd_launches(const LaArgs& a) { return plan_of(a, false).split ? 3 : 1; }

ll_status la_fwd_launch(const LaArgs& a) {
  const Plan pl = plan_of(a, false);
  char* ws = static_cast<char*>(a.ws);
  RecParams p = rec_params(a, pl.seg);
  float* sums = reinterpret_cast<float*>(ws + pl.sum_s);
  ll_status st;
  if (pl.split) {
    p.log_decay = reinterpret_cast<float*>(ws + pl.dec);
    if (pl.tc) {
      st = la_tc_sum_launch(a, pl.seg, pl.slots, 1, sums, nullptr, p.log_decay);
    } else {
      p.job[0] = job_o(a);
      p.job[0].sum = sums;
      st = rec_launch<false>(a.io, a.dk, p, 1, pl.slots, a.stream, false);
    }
    if (st != LL_OK) return st;
    const LaCarry c{p.seqs, pl.seg, (int)elems_of(a), {sums, nullptr}, p.log_decay, {a.state_in, nullptr}};
    st = carry_launch(c, la_sequences(a), a.stream);
    if (st != LL_OK) return st;
    p.log_decay = nullptr;
  }
  const float* in = pl.split ? sums : a.state_in;
  if (pl.tc) return la_tc_fwd_main(a, pl.seg, pl.slots, in, pl.split, pl.split);
  p.job[0] = job_o(a);
  p.job[0].in = in;
  p.job[0].in_by_slot = pl.split;
  p.job[0].out = a.o;
  p.job[0].last = a.state_out;
  return rec_launch<true>(a.io, a.dk, p, 1, pl.slots, a.stream, pl.split);
}

size_t la_bwd_workspace(const LaArgs& a) { return plan_of(a, true).total; }
int la_bwd_launches(const LaArgs& a) {
  const Plan pl = plan_of(a, true);
  return (pl.split ? 2 : 0) + (pl.tc || a.dk == a.dv ? 1 : 2) + 1 + (a.per_head ? 1 : 0);
}

ll_status la_bwd_launch(const LaArgs& a) {
  const Plan pl = plan_of(a, true);
  char* ws = static_cast<char*>(a.ws);
  RecParams p = rec_params(a, pl.seg);
  float* sum_s = reinterpret_cast<float*>(ws + pl.sum_s);
  float* sum_a = reinterpret_cast<float*>(ws + pl.sum_a);
  float* dec = reinterpret_cast<float*>(ws + pl.dec);
  ll_status st;
  if (pl.split) {
    p.log_decay = dec;
    if (pl.tc) {
      st = la_tc_sum_launch(a, pl.seg, pl.slots, 2, sum_s, sum_a, dec);
    } else {
      p.job[0] = job_o(a);
      p.job[0].sum = sum_s;
      p.job[1] = job_dv(a);
      p.job[1].sum = sum_a;
      st = rec_launch<false>(a.io, a.dk, p, 2, pl.slots, a.stream, false);
    }
    if (st != LL_OK) return st;
    const LaCarry c{p.seqs, pl.seg, (int)elems_of(a), {sum_s, sum_a}, dec, {a.state_in, a.dstate_out}};
    st = carry_launch(c, la_sequences(a), a.stream);
    if (st != LL_OK) return st;
    p.log_decay = nullptr;
  }
  const bool own = a.H == a.Hk, chained = pl.split;
  const float* states = pl.split ? sum_s : a.state_in;
  const float* adjoints = pl.split ? sum_a : a.dstate_out;
  // The gradient before a sequence is what its first decay's gradient is made of with the
  // state there, and dstate_in.  In dstate_out's place it has to wait until all have read that.
  const bool aside = !pl.split && a.dstate_in == a.dstate_out;
  float* first = a.dstate_in && !aside ? a.dstate_in : a.dstate_in || a.state_in ? reinterpret_cast<float*>(ws + pl.first) : nullptr;
  // the states behind the sequences, which the last decays' gradients end with where those states have gradients
  float* after = a.dstate_out ? reinterpret_cast<float*>(ws + pl.after) : nullptr;
  float* part_q = reinterpret_cast<float*>(ws + pl.part_q);
  float* part_k = reinterpret_cast<float*>(ws + pl.part_k);
  float* dq32 = own ? nullptr : reinterpret_cast<float*>(ws + pl.dq);
  float* dk32 = own ? nullptr : reinterpret_cast<float*>(ws + pl.dk);
  if (pl.tc) {
    st = la_tc_bwd_main(a, pl.seg, pl.slots, states, adjoints, pl.split, first, after, dq32, dk32, part_q, part_k, chained);
    if (st != LL_OK) return st;
  } else {
    RecJob v = job_dv(a), q{}, k{};
    v.in = adjoints;
    v.in_by_slot = pl.split;
    v.out = a.dval;
    v.last = first;
    q.y = a.k;
    q.z = a.v;
    q.x = a.dout;
    q.w = a.q;
    q.y_key = true;
    q.trans = true;
    q.rows = a.dk;
    q.y_scale = 1.f;
    q.f = a.scale;
    q.in = states;
    q.in_by_slot = pl.split;
    q.out = own ? a.dq : dq32;
    q.out_f32 = !own;
    q.part = part_q;
    k = q;
    q.last = after;
    k.y = a.q;
    k.z = a.dout;
    k.x = a.v;
    k.w = a.k;
    k.rev = true;
    k.y_scale = a.scale;
    k.f = 1.f;
    k.in = adjoints;
    k.out = own ? a.dkey : dk32;
    k.part = part_k;
    p.job[0] = q;
    p.job[1] = k;
    p.job[2] = v;
    st = rec_launch<true>(a.io, a.dv, p, a.dk == a.dv ? 3 : 2, pl.slots, a.stream, chained);
    if (st != LL_OK) return st;
    if (a.dk != a.dv) {
      p.job[0] = v;
      st = rec_launch<true>(a.io, a.dk, p, 1, pl.slots, a.stream, true);
      if (st != LL_OK) return st;
    }
  }
  FinishParams f{};
  f.seqs = p.seqs;
  f.seg = pl.seg;
  f.dk = a.dk;
  f.dv = a.dv;
  f.per_head = a.per_head;
  f.parts = pl.parts;
  f.part_stride = p.part_stride;
  f.log_alpha = a.log_alpha;
  f.part_q = part_q;
  f.part_k = part_k;
  f.entry = states;
  f.by_slot = pl.split;
  f.behind = sum_a;
  f.first = first;
  f.copy_first = aside ? a.dstate_in : nullptr;
  f.after = after;
  f.dstate_out = a.dstate_out;
  f.dlog_alpha = a.dlog_alpha;
  f.head_sums = reinterpret_cast<double*>(ws + pl.heads);
  f.dq = dq32;
  f.dkey = dk32;
  f.dq_out = a.dq;
  f.dk_out = a.dkey;
  const size_t segments = pl.slots * a.H, rows = kFinishThreads / (a.dk / 4);
  f.key_rows = own ? 0u : (unsigned)((size_t)a.B * a.Hk * a.T);
  const size_t grid = segments + (f.key_rows + rows - 1) / rows * 2;
  if (grid > 0x7fffffffull) return LL_ERR_UNSUPPORTED;
  f.segments = (unsigned)segments;
  st = a.io == LL_F32 ? la_launch(true, la_finish_kernel<float>, dim3((unsigned)grid), kFinishThreads, 0, a.stream, f)
                      : la_launch(true, la_finish_kernel<__nv_bfloat16>, dim3((unsigned)grid), kFinishThreads, 0, a.stream, f);
  if (st != LL_OK || !a.per_head) return st;
  const double* sums = f.head_sums;
  return la_launch(true, la_head_sum_kernel, dim3((unsigned)a.H), 128, 0, a.stream, sums, (int)pl.slots, a.H, a.dlog_alpha);
}

}  // namespace llattn

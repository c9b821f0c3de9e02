// The gated delta rule token by token, states in registers: the forward, the
// reverse recurrence of its gradient, and one decode step.
//
// Every row r of a state (d_v) follows a recurrence of its own,
//   e = v[r] - alpha S[r].k,  u = beta e,  S[r] <- alpha S[r] + u k,
//   o[r] = scale S[r].q = scale (alpha S_old[r].q + u k.q),
// so a row needs dot products with the old state and no other row: a group
// of kLpr lanes holds a row (dk / kLpr elements each, four consecutive ones at
// a time so that the lanes of a group read 16- or 8-byte pieces side by side),
// and a CTA 16 rows of one (sequence, head).  Likewise backwards, with C_t the
// adjoint of S_t by the tokens behind t and d = scale do:
//   w = C.k + d q.k,  C <- alpha (C + d q - beta w k).
//
// A token's chain (dot product, sum over the lanes, update) is what bounds these
// kernels, so the sums run one token ahead: S_{t-1}.k_t is
// alpha_{t-1} S_{t-2}.k_t + u_{t-1} k_{t-1}.k_t, whose first product is summed
// while token t - 1 updates the state; likewise backwards.  The products of
// neighbouring keys are made once per staged tile.  Arithmetic is on pairs of
// floats (one instruction for two).  Half of a CTA's threads walk over the tokens;
// the others stage the tile after the next, make the next tile's decays and products of
// neighbours and write the last tile's results, one barrier a tile.  A token takes
// 0.12 us at d_k = 128 (0.075 at 32) while every CTA has an SM's schedulers to
// itself: T = 1001, 8 heads of 32 x 64, float32, 76 us, from 133 with the sums in line.
#include "gdr.cuh"
#include "sm100.cuh"

namespace llattn {

namespace {

using sm100::cp_async16;
using sm100::cp_async_commit;
using sm100::cp_async_wait;
using sm100::named_bar_sync;

constexpr int kRows = 16;    // rows of d_v per CTA
constexpr int kTile = 16;    // tokens staged at a time
static_assert(kGdrGradChunk % kTile == 0, "kept states lie on tile boundaries");
static_assert(kTile % 3 == 1, "the loops over a whole tile take three tokens at a time and one more");

// Lanes per row: fewer make a longer dot product of a lane, more a longer sum
// over the lanes (and threads that share an SM's issue slots).  Measured, forward / gradient in
// us, float32, 512 tokens, 8 and 256 heads: d = 128 with 4 lanes 96 / 171 and 1005 / 3163, with 8
// 69 / 146 and 745 / 2790, with 16 93 / 168 and 1267 / 3605; d = 64 with 2, 4, 8: 81 / 116, 50 / 86, 53 / 92
// and 295 / 1122, 200 / 1040, 247 / 1093; d = 32 with 2, 4, 8: 44 / 65, 42 / 57, 42 / 61 and 84 / 350, 73 / 332,
// 96 / 369; d = 16 with 2, 4: 30 / 44, 31 / 49 and 31 / 160, 41 / 164.
template <int DK> struct RowCfg {
  static constexpr int kLpr = DK >= 128 ? 8 : DK >= 32 ? 4 : 2;  // lanes per row
  static constexpr int kEpl = DK / kLpr;          // elements per lane
  static constexpr int kPieces = kEpl / 4;
  static constexpr int kThreads = kRows * kLpr;
};

// four consecutive elements as float
__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* x) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
}

template <int DK, typename P>
__device__ __forceinline__ void load_row(const P* row, int l, float* x) {
#pragma unroll
  for (int c = 0; c < RowCfg<DK>::kPieces; ++c) load4(row + (c * RowCfg<DK>::kLpr + l) * 4, x + 4 * c);
}
template <int DK>
__device__ __forceinline__ void store_row(float* row, int l, const float* x) {
#pragma unroll
  for (int c = 0; c < RowCfg<DK>::kPieces; ++c)
    *reinterpret_cast<float4*>(row + (c * RowCfg<DK>::kLpr + l) * 4) =
        make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
}
template <int N>
__device__ __forceinline__ float dot(const float* a, const float* b) {
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) s[i & 3] = fmaf(a[i], b[i], s[i & 3]);
  return (s[0] + s[1]) + (s[2] + s[3]);
}
template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
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
__device__ __forceinline__ float sum2(f2 a) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
  return x + y;
}
template <int DK, typename P>
__device__ __forceinline__ void load_pairs(const P* row, int l, f2* x) {
  float y[RowCfg<DK>::kEpl];
  load_row<DK>(row, l, y);
#pragma unroll
  for (int i = 0; i < RowCfg<DK>::kEpl / 2; ++i) x[i] = pair(y[2 * i], y[2 * i + 1]);
}
template <int N>
__device__ __forceinline__ float dot2(const f2* a, const f2* b) {  // of N pairs
  f2 s = mul2(a[0], b[0]), t = mul2(a[1], b[1]);
#pragma unroll
  for (int i = 2; i < N; i += 2) {
    s = fma2(a[i], b[i], s);
    t = fma2(a[i + 1], b[i + 1], t);
  }
  return sum2(s) + sum2(t);
}

// rows [r0, r0 + n) of a [.., W] matrix, W * sizeof(IO) a multiple of 16, into
// shared memory, `cols` columns from column c0, by `threads` threads
template <typename IO>
__device__ __forceinline__ void stage(IO* dst, const IO* src, int n, int width, int c0, int cols, int t, int threads) {
  const int per = cols * (int)sizeof(IO) / 16, el = 16 / (int)sizeof(IO);
  for (int x = t; x < n * per; x += threads) {
    const int r = x / per, p = x - r * per;
    cp_async16(dst + r * cols + p * el, src + (size_t)r * width + c0 + p * el);
  }
}

struct RecParams {
  GdrSeqs seqs;
  int dv;
  float scale;
  const void *q, *k, *v;
  const float *log_alpha, *beta, *state_in;
  void* o;
  float* state_out;
  // for the gradient: the state before every kGdrGradChunk tokens
  // [slot, H, dv, dk] and e [B, H, T, dv]; null otherwise
  float *kept_states, *kept_errors;
  // the reverse recurrence
  const void* dout;
  const float* dstate_out;
  float* dstate_in;
  float *kept_adjoints, *kept_w;
  unsigned* err;
};

// what a tile of tokens needs, three of them in flight
template <typename IO, int DK> struct RecTile {
  IO k[kTile * DK], q[kTile * DK], x[kTile * kRows];  // x: v, or do
};
// results and products of neighbours, two tiles in flight
struct RecSide {
  float4 tok[kTile];
  float more[kTile];
  float out[kTile][kRows], err[kTile][kRows];
};
template <typename IO, int DK> struct RecSm {
  RecTile<IO, DK> tile[3];
  RecSide side[2];
};
constexpr int kHelpBar = 1;

// The decays of a tile's tokens (lane t's is `la` of token t; whole warp), from the last one back if
// REV.  A state is multiplied by one after another, so that a rounding that repeats (0.9999, token
// after token) would add up over its memory: what the product so far is off by, `off` (relative), is
// taken out of the next factor before that is rounded, and the product of any run of them is within
// a few roundings of the exact one.  exp(la) - 1 keeps a factor near 1 exact until it is rounded; those
// that are not leave `off` to the next one.  It takes 300 cycles a tile, beside the recurrence.
template <bool REV> __device__ __forceinline__ float tile_decays(float la, float& off, int lane) {
  const bool near = la > -0.5f;
  const float m = near ? expm1f(la) : 0.f;
  float own = 0.f;
#pragma unroll
  for (int x = 0; x < kTile; ++x) {
    const int t = REV ? kTile - 1 - x : x;
    const float c = __shfl_sync(0xffffffffu, m, t) - off, r = 1.f + c;
    off = (r - 1.f) - c;
    if (lane == t) own = r;
  }
  return near ? own : expf(la);
}

// The recurrence.
template <typename IO, int DK>
__device__ __forceinline__ void rec_forward(const RecParams& p) {
  using Cfg = RowCfg<DK>;
  constexpr int LPR = Cfg::kLpr, NP = Cfg::kEpl / 2, NT = Cfg::kThreads;
  extern __shared__ __align__(16) unsigned char raw[];
  RecSm<IO, DK>& sm = *reinterpret_cast<RecSm<IO, DK>*>(raw);

  const int slices = p.dv / kRows;
  const int sl = blockIdx.x % slices;
  const int h = (blockIdx.x / slices) % p.seqs.H;
  const int seq = gdr_pick(p.seqs, blockIdx.x / slices / p.seqs.H);
  const bool helper = threadIdx.x >= NT;
  const int tid = threadIdx.x % NT, grp = tid / LPR, l = tid % LPR;
  const int r0 = sl * kRows;
  GdrSeq sq;
  if (!gdr_seq(p.seqs, seq, sq)) {
    if (threadIdx.x == 0) raise_error(p.err, kErrDeviceArg);
    return;
  }
  const int hk = h / (p.seqs.H / p.seqs.Hk);
  const size_t row0 = ((size_t)sq.row_b * p.seqs.H + h) * p.seqs.T + sq.start;
  const size_t krow0 = ((size_t)sq.row_b * p.seqs.Hk + hk) * p.seqs.T + sq.start;
  const int tiles = (sq.len + kTile - 1) / kTile;

  if (helper) {
    const IO* qg = static_cast<const IO*>(p.q) + krow0 * DK;
    const IO* kg = static_cast<const IO*>(p.k) + krow0 * DK;
    const IO* vg = static_cast<const IO*>(p.v) + row0 * p.dv;
    IO* og = p.o ? static_cast<IO*>(p.o) + row0 * p.dv : nullptr;
    float la = 0.f, bt = 0.f, off = 0.f;
    auto fetch = [&](int j) {  // (one group of copies a tile, an empty one behind the last)
      if (j < tiles) {
        const int t0 = j * kTile, n = min(kTile, sq.len - t0);
        RecTile<IO, DK>& t = sm.tile[j % 3];
        stage(t.k, kg + (size_t)t0 * DK, n, DK, 0, DK, tid, NT);
        stage(t.q, qg + (size_t)t0 * DK, n, DK, 0, DK, tid, NT);
        stage(t.x, vg + (size_t)t0 * p.dv, n, p.dv, r0, kRows, tid, NT);
      }
      cp_async_commit();
    };
    auto gates = [&](int j) {
      const int t = j * kTile + grp, ta = j * kTile + tid;
      if (l == 0 && t < sq.len) bt = p.beta[row0 + t];
      if (tid < kTile) la = ta < sq.len ? p.log_alpha[row0 + ta] : 0.f;
    };
    // tile j: its decays and, once it is there, its products of neighbours, one group of lanes to a token
    auto products = [&](int j) {
      float4* tok = sm.side[j & 1].tok;
      if (tid < 32) {
        const float d = tile_decays<false>(la, off, tid);
        if (tid < kTile) tok[tid].x = d;
      }
      cp_async_wait<1>();
      named_bar_sync(kHelpBar, NT);
      const RecTile<IO, DK>& t = sm.tile[j % 3];
      f2 x[NP], y[NP];
      load_pairs<DK>(t.k + grp * DK, l, x);
      load_pairs<DK>(t.q + grp * DK, l, y);
      const float kq = group_sum<LPR>(dot2<NP>(x, y));
      load_pairs<DK>(t.k + max(grp - 1, 0) * DK, l, y);
      const float kk = group_sum<LPR>(dot2<NP>(x, y));
      if (l == 0) {
        tok[grp].y = bt;
        tok[grp].z = kq;
        tok[grp].w = kk;
      }
      gates(j + 1);  // (on their way until the next tile's products)
    };
    gates(0);
    fetch(0);
    fetch(1);
    if (tiles) products(0);
    __syncthreads();
    for (int j = 0; j <= tiles; ++j) {
      if (j > 0) {  // the results of tile j - 1
        const int t0 = (j - 1) * kTile, n = min(kTile, sq.len - t0);
        const RecSide& side = sm.side[(j - 1) & 1];
        for (int x = tid; x < n * kRows; x += NT) {
          const int t = x / kRows, r = x % kRows;
          const size_t at = (size_t)(t0 + t) * p.dv + r0 + r;
          if (og) og[at] = from_f<IO>(side.out[t][r]);
          if (p.kept_errors) p.kept_errors[row0 * p.dv + at] = side.err[t][r];
        }
      }
      fetch(j + 2);
      if (j + 1 < tiles) products(j + 1);
      __syncthreads();
    }
    cp_async_wait<0>();
    return;
  }

  const size_t st_at = (((size_t)seq * p.seqs.H + h) * p.dv + r0 + grp) * DK;
  const int base = gdr_slot_base(p.seqs, seq, sq.start, kGdrGradChunk);
  f2 s[NP];
  if (p.state_in) load_pairs<DK>(p.state_in + st_at, l, s);
  else
#pragma unroll
    for (int i = 0; i < NP; ++i) s[i] = 0;
  __syncthreads();
  for (int j = 0; j < tiles; ++j) {
    const int t0 = j * kTile, n = min(kTile, sq.len - t0);
    const RecTile<IO, DK>& tl = sm.tile[j % 3];
    RecSide& side = sm.side[j & 1];
    if (p.kept_states && t0 % kGdrGradChunk == 0)
      store_row<DK>(p.kept_states +
                        ((((size_t)base + t0 / kGdrGradChunk) * p.seqs.H + h) * p.dv + r0 + grp) * DK, l,
                    reinterpret_cast<const float*>(s));
    // one token's work, its operands loaded before; k2 and q1 are loaded for the tokens ahead
    f2 ka[NP], kb[NP], kc[NP], qa[NP], qb[NP];
    load_pairs<DK>(tl.k, l, ka);
    load_pairs<DK>(tl.k + min(1, kTile - 1) * DK, l, kb);
    load_pairs<DK>(tl.q, l, qa);
    float4 c = side.tok[0];
    float v = to_f(tl.x[grp]);
    float dn = group_sum<LPR>(dot2<NP>(s, ka));  // of the state one token back (here: the present one) with this key
    float a_p = 1.f, u_p = 0.f;
    auto token = [&](int t, f2* k0, f2* k1, f2* k2, f2* q0, f2* q1) {
      float d1 = dot2<NP>(s, k1), d2 = dot2<NP>(s, q0);
      const float e = fmaf(-c.x, fmaf(a_p, dn, c.w * u_p), v);
      const float u = c.y * e;
      const float al_t = c.x, kq_t = c.z;
      const int t1 = min(t + 1, kTile - 1);
      c = side.tok[t1];
      v = to_f(tl.x[t1 * kRows + grp]);
      load_pairs<DK>(tl.k + min(t + 2, kTile - 1) * DK, l, k2);
      load_pairs<DK>(tl.q + t1 * DK, l, q1);
      const f2 a2 = pair(al_t, al_t), u2 = pair(u, u);
#pragma unroll
      for (int i = 0; i < NP; ++i) s[i] = fma2(u2, k0[i], mul2(a2, s[i]));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) {
        d1 += __shfl_xor_sync(0xffffffffu, d1, o);
        d2 += __shfl_xor_sync(0xffffffffu, d2, o);
      }
      if (l == 0) {
        side.out[t][grp] = p.scale * fmaf(al_t, d2, u * kq_t);
        side.err[t][grp] = e;
      }
      dn = d1;
      a_p = al_t;
      u_p = u;
    };
    if (n == kTile) {  // (the operands change places, no copies)
#pragma unroll 1
      for (int t = 0; t < kTile - 1; t += 3) {
        token(t, ka, kb, kc, qa, qb);
        token(t + 1, kb, kc, ka, qb, qa);
        token(t + 2, kc, ka, kb, qa, qb);
#pragma unroll
        for (int i = 0; i < NP; ++i) qa[i] = qb[i];
      }
      token(kTile - 1, ka, kb, kc, qa, qb);
    } else {
#pragma unroll 1
      for (int t = 0; t < n; ++t) {
        token(t, ka, kb, kc, qa, qb);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          ka[i] = kb[i];
          kb[i] = kc[i];
          qa[i] = qb[i];
        }
      }
    }
    __syncthreads();
  }
  __syncthreads();
  if (p.state_out) store_row<DK>(p.state_out + st_at, l, reinterpret_cast<const float*>(s));
}

// The reverse recurrence: w_t for every token, the adjoint C behind every
// kGdrGradChunk tokens, and the gradient of the state on entry.  Step x takes
// tile tiles - 1 - x.
template <typename IO, int DK>
__device__ __forceinline__ void rec_reverse(const RecParams& p) {
  using Cfg = RowCfg<DK>;
  constexpr int LPR = Cfg::kLpr, NP = Cfg::kEpl / 2, NT = Cfg::kThreads;
  extern __shared__ __align__(16) unsigned char raw[];
  RecSm<IO, DK>& sm = *reinterpret_cast<RecSm<IO, DK>*>(raw);

  const int slices = p.dv / kRows;
  const int sl = blockIdx.x % slices;
  const int h = (blockIdx.x / slices) % p.seqs.H;
  const int seq = gdr_pick(p.seqs, blockIdx.x / slices / p.seqs.H);
  const bool helper = threadIdx.x >= NT;
  const int tid = threadIdx.x % NT, grp = tid / LPR, l = tid % LPR;
  const int r0 = sl * kRows;
  GdrSeq sq;
  if (!gdr_seq(p.seqs, seq, sq)) {
    if (threadIdx.x == 0) raise_error(p.err, kErrDeviceArg);
    return;
  }
  const int hk = h / (p.seqs.H / p.seqs.Hk);
  const size_t row0 = ((size_t)sq.row_b * p.seqs.H + h) * p.seqs.T + sq.start;
  const size_t krow0 = ((size_t)sq.row_b * p.seqs.Hk + hk) * p.seqs.T + sq.start;
  const int tiles = (sq.len + kTile - 1) / kTile;

  if (helper) {
    const IO* qg = static_cast<const IO*>(p.q) + krow0 * DK;
    const IO* kg = static_cast<const IO*>(p.k) + krow0 * DK;
    const IO* dg = static_cast<const IO*>(p.dout) + row0 * p.dv;
    float la = 0.f, bt = 0.f, off = 0.f;
    auto fetch = [&](int x) {
      if (x < tiles) {
        const int t0 = (tiles - 1 - x) * kTile, n = min(kTile, sq.len - t0);
        RecTile<IO, DK>& t = sm.tile[x % 3];
        stage(t.k, kg + (size_t)t0 * DK, n, DK, 0, DK, tid, NT);
        stage(t.q, qg + (size_t)t0 * DK, n, DK, 0, DK, tid, NT);
        stage(t.x, dg + (size_t)t0 * p.dv, n, p.dv, r0, kRows, tid, NT);
      }
      cp_async_commit();
    };
    auto gates = [&](int x) {
      const int t = (tiles - 1 - x) * kTile + grp, ta = (tiles - 1 - x) * kTile + tid;
      if (l == 0 && x < tiles && t < sq.len) bt = p.beta[row0 + t];
      if (tid < kTile) la = x < tiles && ta < sq.len ? p.log_alpha[row0 + ta] : 0.f;
    };
    auto products = [&](int x) {
      float4* tok = sm.side[x & 1].tok;
      if (tid < 32) {
        const float d = tile_decays<true>(la, off, tid);
        if (tid < kTile) tok[tid].x = d;
      }
      cp_async_wait<1>();
      named_bar_sync(kHelpBar, NT);
      const RecTile<IO, DK>& t = sm.tile[x % 3];
      f2 a[NP], b[NP], z[NP];
      load_pairs<DK>(t.k + grp * DK, l, a);
      load_pairs<DK>(t.q + grp * DK, l, b);
      load_pairs<DK>(t.k + max(grp - 1, 0) * DK, l, z);
      const float qk = group_sum<LPR>(dot2<NP>(a, b)), qk1 = group_sum<LPR>(dot2<NP>(b, z));
      const float kk = group_sum<LPR>(dot2<NP>(a, z));
      if (l == 0) {
        tok[grp].y = bt;
        tok[grp].z = qk;
        tok[grp].w = qk1;
        sm.side[x & 1].more[grp] = kk;
      }
      gates(x + 1);
    };
    gates(0);
    fetch(0);
    fetch(1);
    if (tiles) products(0);
    __syncthreads();
    for (int x = 0; x <= tiles; ++x) {
      if (x > 0) {
        const int t0 = (tiles - x) * kTile, n = min(kTile, sq.len - t0);
        const RecSide& side = sm.side[(x - 1) & 1];
        for (int e = tid; e < n * kRows; e += NT) {
          const int t = e / kRows, r = e % kRows;
          p.kept_w[(row0 + t0 + t) * p.dv + r0 + r] = side.out[t][r];
        }
      }
      fetch(x + 2);
      if (x + 1 < tiles) products(x + 1);
      __syncthreads();
    }
    cp_async_wait<0>();
    return;
  }

  const size_t st_at = (((size_t)seq * p.seqs.H + h) * p.dv + r0 + grp) * DK;
  const int base = gdr_slot_base(p.seqs, seq, sq.start, kGdrGradChunk);
  f2 a[NP];
  if (p.dstate_out) load_pairs<DK>(p.dstate_out + st_at, l, a);
  else
#pragma unroll
    for (int i = 0; i < NP; ++i) a[i] = 0;
  __syncthreads();
  for (int x = 0; x < tiles; ++x) {
    const int t0 = (tiles - 1 - x) * kTile, n = min(kTile, sq.len - t0);
    const RecTile<IO, DK>& tl = sm.tile[x % 3];
    RecSide& side = sm.side[x & 1];
    if (t0 + n == sq.len || (t0 + n) % kGdrGradChunk == 0)
      store_row<DK>(p.kept_adjoints +
                        ((((size_t)base + t0 / kGdrGradChunk) * p.seqs.H + h) * p.dv + r0 + grp) * DK, l,
                    reinterpret_cast<const float*>(a));
    f2 ka[NP], kb[NP], kc[NP], qa[NP], qb[NP];
    load_pairs<DK>(tl.k + (n - 1) * DK, l, ka);
    load_pairs<DK>(tl.k + max(n - 2, 0) * DK, l, kb);
    load_pairs<DK>(tl.q + (n - 1) * DK, l, qa);
    float4 c = side.tok[n - 1];
    float kk = side.more[n - 1], d = p.scale * to_f(tl.x[(n - 1) * kRows + grp]);
    float ck = group_sum<LPR>(dot2<NP>(a, ka));  // C_t.k_t
    auto token = [&](int t, f2* k0, f2* k1, f2* k2, f2* q0, f2* q1) {
      float d1 = dot2<NP>(a, k1);
      const float w = fmaf(d, c.z, ck);
      const float bw = -c.y * w, al_t = c.x;
      const float rest = fmaf(d, c.w, bw * kk);
      const f2 al2 = pair(al_t, al_t), d2 = pair(d, d), w2 = pair(bw, bw);
      const int t1 = max(t - 1, 0);
      c = side.tok[t1];
      kk = side.more[t1];
      d = p.scale * to_f(tl.x[t1 * kRows + grp]);
      load_pairs<DK>(tl.k + max(t - 2, 0) * DK, l, k2);
      load_pairs<DK>(tl.q + t1 * DK, l, q1);
#pragma unroll
      for (int i = 0; i < NP; ++i) a[i] = mul2(al2, fma2(w2, k0[i], fma2(d2, q0[i], a[i])));
      d1 = group_sum<LPR>(d1);
      ck = al_t * (d1 + rest);
      if (l == 0) side.out[t][grp] = w;
    };
    if (n == kTile) {
#pragma unroll 1
      for (int t = kTile - 1; t > 0; t -= 3) {
        token(t, ka, kb, kc, qa, qb);
        token(t - 1, kb, kc, ka, qb, qa);
        token(t - 2, kc, ka, kb, qa, qb);
#pragma unroll
        for (int i = 0; i < NP; ++i) qa[i] = qb[i];
      }
      token(0, ka, kb, kc, qa, qb);
    } else {
#pragma unroll 1
      for (int t = n - 1; t >= 0; --t) {
        token(t, ka, kb, kc, qa, qb);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          ka[i] = kb[i];
          kb[i] = kc[i];
          qa[i] = qb[i];
        }
      }
    }
    __syncthreads();
  }
  __syncthreads();
  if (p.dstate_in) store_row<DK>(p.dstate_in + st_at, l, reinterpret_cast<const float*>(a));
}

template <typename IO, int DK>
__global__ void __launch_bounds__(2 * RowCfg<DK>::kThreads) gdr_rec_fwd_kernel(RecParams p) {
  rec_forward<IO, DK>(p);
}
// For the gradient both at once: neither needs the other, and a sequence's chain
// bounds each (y = 0: the recurrence, y = 1: the reverse one).
template <typename IO, int DK>
__global__ void __launch_bounds__(2 * RowCfg<DK>::kThreads) gdr_rec_both_kernel(RecParams p) {
  if (blockIdx.y == 0) rec_forward<IO, DK>(p);
  else rec_reverse<IO, DK>(p);
}

// ---------------------------------------------------------------- one decode step
// Rows in flight per group of lanes.  Measured with 1, 2 and 4 (128 x 128): 32 states 3.2, 3.1 and 3.8
// us, 256 states 6.8, 6.2 and 6.3, 2048 states 44.8, 44.7 and 44.9.
constexpr int kStepPasses = 2;

// Per (b, h): the state is read and written once, which is what bounds the
// step.  A group of lanes takes kStepPasses rows, all their loads issued
// before any is used; 16 * kStepPasses rows of d_v to a CTA, so that one
// request of few heads still spreads over the SMs.  268 MB (2048 states of 128 x 128)
// in 47 us behind a flushed L2, 85 % of a copy's rate; 885 MB in 141 us, 93 %.
template <typename IO, int DK>
__global__ void __launch_bounds__(RowCfg<DK>::kThreads) gdr_decode_kernel(
    int H, int Hk, int dv, float scale, const int64_t* __restrict__ slots, int n_slots, const IO* __restrict__ q,
    const IO* __restrict__ k, const IO* __restrict__ v, const float* __restrict__ log_alpha,
    const float* __restrict__ beta, float* __restrict__ states, IO* __restrict__ o, unsigned* __restrict__ err) {
  using Cfg = RowCfg<DK>;
  constexpr int LPR = Cfg::kLpr, EPL = Cfg::kEpl;
  __shared__ float os[kRows * kStepPasses];
  const int cta_rows = kRows * kStepPasses;
  const int slices = (dv + cta_rows - 1) / cta_rows;
  const int sl = blockIdx.x % slices;
  const int h = (blockIdx.x / slices) % H;
  const int b = blockIdx.x / slices / H;
  const int tid = threadIdx.x, grp = tid / LPR, l = tid % LPR;
  const size_t bh = (size_t)b * H + h;
  const size_t bk = (size_t)b * Hk + h / (H / Hk);
  long long slot = slots ? slots[b] : b;
  float kv[EPL], qv[EPL];
  load_row<DK>(k + bk * DK, l, kv);
  load_row<DK>(q + bk * DK, l, qv);
  const float la = log_alpha[bh], be = beta[bh];
  if (slot < 0 || slot >= n_slots) {  // -1 is a row of padding; anything else out of range an error
    if (slot != -1 && tid == 0) raise_error(err, kErrDeviceArg);
    return;
  }
  float* st = states + ((size_t)slot * H + h) * dv * DK;
  float s[kStepPasses][EPL], vv[kStepPasses];
  const int r0 = sl * cta_rows + grp;
#pragma unroll
  for (int x = 0; x < kStepPasses; ++x) {
    const int r = r0 + kRows * x;
    if (r < dv) {
      load_row<DK>(st + (size_t)r * DK, l, s[x]);
      vv[x] = to_f(v[bh * dv + r]);
    }
  }
  // two rows of the batch with one slot would race: one CTA of the row looks
  if (slots && sl == 0 && h == 0)
    for (int x = tid; x < b; x += Cfg::kThreads)
      if (slots[x] == slot) raise_error(err, kErrDeviceArg);
  // alpha x, near 1 as x + (alpha - 1) x: step after step a rounded alpha would add up over the state's memory
  const bool near = la > -0.5f;
  const float a = near ? expm1f(la) : expf(la);
  auto decayed = [&](float x) { return fmaf(a, x, near ? x : 0.f); };
  const bool forget = a == 0.f && !near;  // whatever the state holds: slots are handed on
  const float c = group_sum<LPR>(dot<EPL>(kv, qv));
#pragma unroll
  for (int x = 0; x < kStepPasses; ++x) {
    const int r = r0 + kRows * x;
    float sk = 0.f, sqd = 0.f;
    if (r < dv) {
      if (forget)
#pragma unroll
        for (int i = 0; i < EPL; ++i) s[x][i] = 0.f;
      sk = dot<EPL>(s[x], kv);
      sqd = dot<EPL>(s[x], qv);
    }
    sk = group_sum<LPR>(sk);
    sqd = group_sum<LPR>(sqd);
    if (r < dv) {
      const float u = be * (vv[x] - decayed(sk));
#pragma unroll
      for (int i = 0; i < EPL; ++i) s[x][i] = fmaf(u, kv[i], decayed(s[x][i]));
      store_row<DK>(st + (size_t)r * DK, l, s[x]);
      if (l == 0) os[grp + kRows * x] = scale * fmaf(u, c, decayed(sqd));
    }
  }
  __syncthreads();
  if (tid < cta_rows && sl * cta_rows + tid < dv) o[bh * dv + sl * cta_rows + tid] = from_f<IO>(os[tid]);
}

template <template <typename, int> class F, typename... A>
ll_status by_type(ll_dtype io, int dk, A... args) {
  const bool f = io == LL_F32;
  switch (dk) {
    case 16: return f ? F<float, 16>::run(args...) : F<__nv_bfloat16, 16>::run(args...);
    case 32: return f ? F<float, 32>::run(args...) : F<__nv_bfloat16, 32>::run(args...);
    case 64: return f ? F<float, 64>::run(args...) : F<__nv_bfloat16, 64>::run(args...);
    case 128: return f ? F<float, 128>::run(args...) : F<__nv_bfloat16, 128>::run(args...);
  }
  return LL_ERR_UNSUPPORTED;
}

template <typename IO, int DK> struct Rec {
  static ll_status run(const RecParams& p, unsigned grid, bool both, cudaStream_t st) {
    constexpr int smem = (int)sizeof(RecSm<IO, DK>);
    auto kernel = both ? gdr_rec_both_kernel<IO, DK> : gdr_rec_fwd_kernel<IO, DK>;
    if (smem > 48 * 1024) LL_CUDA_OK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    kernel<<<dim3(grid, both ? 2 : 1), 2 * RowCfg<DK>::kThreads, smem, st>>>(p);
    LL_CUDA_OK(cudaGetLastError());
    return LL_OK;
  }
};

RecParams rec_params(const GdrArgs& a) {
  RecParams p{};
  p.seqs = GdrSeqs{a.n_seqs ? a.seq_starts : nullptr, gdr_sequences(a), a.T, a.H, a.Hk};
  p.dv = a.dv;
  p.scale = a.scale;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.log_alpha = a.log_alpha;
  p.beta = a.beta;
  p.state_in = a.state_in;
  p.err = a.err;
  return p;
}
unsigned rec_grid(const GdrArgs& a) { return (unsigned)((size_t)gdr_sequences(a) * a.H * (a.dv / kRows)); }

}  // namespace

ll_status gdr_rec_fwd_launch(const GdrArgs& a) {
  RecParams p = rec_params(a);
  p.o = a.o;
  p.state_out = a.state_out;
  return by_type<Rec, const RecParams&, unsigned, bool, cudaStream_t>(a.io, a.dk, p, rec_grid(a), false, a.stream);
}

ll_status gdr_rec_both_launch(const GdrArgs& a, float* kept_states, float* kept_errors, float* kept_adjoints,
                              float* kept_w) {
  RecParams p = rec_params(a);
  p.kept_states = kept_states;
  p.kept_errors = kept_errors;
  p.dout = a.dout;
  p.dstate_out = a.dstate_out;
  p.dstate_in = a.dstate_in;
  p.kept_adjoints = kept_adjoints;
  p.kept_w = kept_w;
  return by_type<Rec, const RecParams&, unsigned, bool, cudaStream_t>(a.io, a.dk, p, rec_grid(a), true, a.stream);
}

namespace {
struct StepArgs {
  int B, H, Hk, dv;
  float scale;
  const int64_t* slots;
  int n_slots;
  const void *q, *k, *v;
  const float *la, *beta;
  float* states;
  void* o;
  cudaStream_t stream;
  unsigned* err;
};
template <typename IO, int DK> struct Step {
  static ll_status run(const StepArgs& a) {
    const int rows = kRows * kStepPasses;
    const unsigned grid = (unsigned)((size_t)a.B * a.H * ((a.dv + rows - 1) / rows));
    gdr_decode_kernel<IO, DK><<<grid, RowCfg<DK>::kThreads, 0, a.stream>>>(
        a.H, a.Hk, a.dv, a.scale, a.slots, a.n_slots, static_cast<const IO*>(a.q), static_cast<const IO*>(a.k),
        static_cast<const IO*>(a.v), a.la, a.beta, a.states, static_cast<IO*>(a.o), a.err);
    LL_CUDA_OK(cudaGetLastError());
    return LL_OK;
  }
};
}  // namespace

ll_status gdr_decode_launch(int B, int H, int Hk, int dk, int dv, ll_dtype io, float scale, const int64_t* slots,
                            int n_slots, const void* q, const void* k, const void* v, const float* log_alpha,
                            const float* beta, float* states, void* o, cudaStream_t stream, unsigned* err) {
  const StepArgs a{B, H, Hk, dv, scale, slots, n_slots, q, k, v, log_alpha, beta, states, o, stream, err};
  return by_type<Step, const StepArgs&>(io, dk, a);
}

}  // namespace llattn

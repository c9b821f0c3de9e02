// Linear attention with a decay per head on the tensor cores, in chunks of 128
// tokens: bf16 io, head sizes of 64 and 128.
//
// The forward and the three gradients are one computation with different roles
// (la_rec.cu): with scores P = q k^T . decays (masked to the past, backwards to the
// future) and M the state at the chunk's border,
//   out = scale P v + exp(log decay from the border) q M^T,
//   M <- exp(chunk's log decay) M + v^T diag(weights) k,
//   o    q = Q,   k = K,   v = V,   M = S       forwards
//   dq   q = dO,  k = V,   v = K,   M = S^T     forwards
//   dk   q = V,   k = dO,  v = Q,   M = A^T     backwards
//   dv   q = K,   k = Q,   v = dO,  M = A       backwards
// Five products of 128 x 128 x 128 a chunk: q k^T, q M^T, P v and v^T k' of two parts; six of three.
//
// Precision.  States (and their gradients) that leave the call are float32 results: k' = weight k goes
// into their products in three bf16 parts, all of float32's 24 bits (1.5e-7 of a state's norm; with two it was
// 2.5e-6).  A state that goes no further than o, which is rounded to bf16, has two.  P and the state
// in q M^T are rounded to bf16 once, as the output is.  Where the decay's gradient is made of the states (dq, dv and
// their segments' sums), k' and the state in q M^T have three parts, and what lies within
// the chunk is summed in float32 from two tiles of scores: sum_j P_ij (w v^T)_ij with w = Q (V).  (Two parts of the
// state: 2.2e-6 of d log alpha at B 2, H 16, T 4096, three 3.3e-7; 9 us of 216, since the high part waits for
// the least one's product in its place.)
// bf16 has float32's range, so no operand is scaled.
//
// Bound: the chain of a chunk, 2.7 us of which the products take half (the scores' masking and k' stand between
// them).  More segments are more chunks at a time: a pass
// that sums up what each adds to the state, one along them, then all of them at once.  B 2, H 16, T 4096, d 128:
// 65 us a call (sums 24, carry 7, outputs 39; 20 at the copy rate), its gradient 216 (sums 34, carry 9, dq dk dv 167, decays 14).
//
// Decays between two tokens of a chunk are products of factors of at most 1: from the
// row to its block of 32, over the blocks between, from the column's block to the column;
// only the 32 x 32 blocks on the diagonal take an exponential per element.
#include <algorithm>
#include <atomic>
#include <cmath>

#include <cudaTypedefs.h>

#include "gdr_tc.cuh"
#include "la.cuh"

namespace llattn {
namespace {

using namespace gdrtc;

// Bounded wait, as a call.
static __device__ __noinline__ void wait_at(uint32_t bar, uint32_t par, unsigned* err) {
  const uint64_t t0 = globaltimer_ns();
  uint32_t ok;
  do {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(par)
        : "memory");
    if (!ok && globaltimer_ns() - t0 > kTimeoutNs) {
      atomicOr(err, kErrTimeout);
      return;
    }
  } while (!ok);
}
__device__ __forceinline__ bool try_wait_at(uint32_t bar, uint32_t par) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(par)
      : "memory");
  return ok != 0;
}
// A group waits by one of its warps, the others at a named barrier: twenty warps that poll took most of
// the issue slots, and the products and the scores beside them twice their time (18 thousand cycles a chunk
// of dq or dv with them).
#define LL_GROUP_WAIT(leads, id, threads, waits) \
  do {                                           \
    if (leads) {                                 \
      waits;                                     \
    }                                            \
    named_bar_sync(id, threads);                 \
  } while (0)

// ---- parameters
struct TcJob {
  const float* in;      // states on entry, by slot or by sequence; null: zero
  float* last;          // the state behind the sequence (backwards: before it), or null
  bool in_by_slot;
  float* out_f32;       // [B,H,T,DY] float32 in the place of `out` (heads are summed later), or null
  float* part;          // [2][B,H,T]: row products for the decay's gradient (halves of the columns), or null
  void* out;            // bf16, for the rows of partial chunks
};
struct TcParams {
  GdrSeqs seqs;
  int seg, per_head, dk, dv;
  float scale;
  size_t part_stride;   // B H T
  const float* log_alpha;
  unsigned* err;
  TcJob job[3];
};
// [rows, d] bf16, boxes of 64 columns and 128 rows
struct FwdMaps {
  CUtensorMap q, k, v, o;
};
struct BwdMaps {
  CUtensorMap q, k, v, dout, dq, dk, dv;
};

// Two groups of warps: eight mask the scores and write the outputs, two threads to a row;
// sixteen hold the state in registers and make k', four to a row.  Warp 24 issues
// the products, 25 the loads, 26 the stores, 27 makes the next chunk's decays.
constexpr int kRowThreads = 256, kStateThreads = 512;
constexpr int kStateWarp = kRowThreads / 32, kIssueWarp = kStateWarp + kStateThreads / 32;
constexpr int kThreads = kRowThreads + kStateThreads + 128;
constexpr int kBufs = 7;
constexpr int kBarRows = 1, kBarState = 2;  // named barriers of the groups

struct Sm {
  static constexpr uint32_t kLog = kBufs * kTile;            // behind the tiles, the chunk's decays: Tab
  static constexpr uint32_t kBars = kLog + 2624;
  static constexpr uint32_t kSlot = kBars + (2 * kBufs + 13) * 8;
  static constexpr uint32_t kBytes = kSlot + 16;
};
static_assert(Sm::kBytes <= 232448, "shared memory budget of one CTA");
enum Bar : int { kFull = 0, kEmpty = kBufs, kS1 = 2 * kBufs, kS2, kS3, kS4, kMb, kP, kKp, kTab, kRead, kStaged, kStored, kLeast, kMhi, kNumBars };
static_assert(kNumBars <= 2 * kBufs + 13, "room for the barriers");

// The log decays of a chunk are summed as integers of 2^-36, exactly, so that a
// sum over the rest of a block is a difference, and one of far smaller ones behind a large
// one loses nothing.  (They are cut off at +-1e4, where their exponentials are 0 and infinite.)
constexpr float kUnit = 1.4551915228366852e-11f;  // 2^-36
__device__ __forceinline__ float log_float(long long x) { return __ll2float_rn(x) * kUnit; }
// times log2(e), as a pair of floats
__device__ __forceinline__ float2 log2_pair(long long x, float bad) {
  constexpr float kLow = 1.9259629911266175e-8f;  // log2(e) = kLog2e + kLow
  const float f = __ll2float_rn(x), hi = f * kUnit, lo = log_float(x - (long long)f);
  const float y = hi * kLog2e;
  return make_float2(y + bad, fmaf(hi, kLog2e, -y) + fmaf(hi, kLow, lo * kLog2e));
}
// What the groups need of a chunk's decays.  A NaN makes all of them NaN.
struct Tab {
  float2 in_block[kC];  // from the block of 32's first token to this one, inclusive; times log2(e), as pairs
  float col[kC];        // the factor of a column: from behind it to its block's end (backwards: from the start to it)
  float c1[kC];         // of a row of q M^T
  float weight[kC];     // of a row of k'
  float2 blk[4];        // the blocks', likewise
  float2 decay;         // of the state: M <- x M + y M
};
static_assert(sizeof(Tab) <= 2624, "");
// One warp, four neighbouring tokens to a lane; la: theirs
struct ChunkLog {
  long long past[4];    // from the chunk's first token to this one, inclusive
  long long first, sum; // in front of this lane's block; of the block
  long long total;
  float bad;            // 0, or NaN
};
__device__ __forceinline__ ChunkLog chunk_log(const float* la, int lane) {
  ChunkLog g;
  bool nan = false;
  long long x = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    nan = nan || la[e] != la[e];
    x += __float2ll_rn(fminf(la[e], 1e4f) * 68719476736.f);
    g.past[e] = x;
  }
  long long y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) g.past[e] += y - x;
  g.first = __shfl_sync(0xffffffffu, y - x, lane & 24);
  g.sum = __shfl_sync(0xffffffffu, y, lane | 7) - g.first;
  g.total = __shfl_sync(0xffffffffu, y, 31);
  g.bad = __any_sync(0xffffffffu, nan) ? __int_as_float(0x7fffffff) : 0.f;
  return g;
}
// a token's entries (an absent token's weight is zero)
struct TabEntry {
  float2 in_block;
  float col, c1, weight;
};
template <bool REV>
__device__ __forceinline__ TabEntry make_entry(const ChunkLog& g, long long past, bool there, float scale) {
  TabEntry t;
  const long long block = past - g.first;
  const float to = expf(log_float(past) + g.bad), from = expf(log_float(g.total - past) + g.bad);
  t.in_block = log2_pair(block, g.bad);
  t.col = ex2(REV ? t.in_block.x : log_float(g.sum - block) * kLog2e) + g.bad;
  t.c1 = REV ? from : scale * to;
  t.weight = !there ? 0.f : REV ? scale * to : from;
  return t;
}
__device__ __forceinline__ void store_whole(Tab* tab, const ChunkLog& g, int lane) {
  if ((lane & 7) == 0) tab->blk[lane >> 3] = log2_pair(g.sum, g.bad);
  if (lane == 0) {
    const LaDecay d = la_decay(log_float(g.total) + g.bad);
    tab->decay = make_float2(d.f, d.near ? 1.f : 0.f);
  }
}
// Made at once, or (SHORT) one after another once the groups are done with the last ones.
template <bool REV>
__device__ __forceinline__ void store_short(Tab* tab, const ChunkLog& g, int lane, int n, float scale) {
#pragma unroll 1
  for (int e = 0; e < 4; ++e) {
    const int i = 4 * lane + e;
    const TabEntry t = make_entry<REV>(g, e == 0 ? g.past[0] : e == 1 ? g.past[1] : e == 2 ? g.past[2] : g.past[3], i < n, scale);
    tab->in_block[i] = t.in_block;
    tab->col[i] = t.col;
    tab->c1[i] = t.c1;
    tab->weight[i] = t.weight;
  }
  store_whole(tab, g, lane);
}
__device__ __forceinline__ void store_tab(Tab* tab, const TabEntry* t, const ChunkLog& g, int lane) {
  float4* p = reinterpret_cast<float4*>(tab->in_block + 4 * lane);
  p[0] = make_float4(t[0].in_block.x, t[0].in_block.y, t[1].in_block.x, t[1].in_block.y);
  p[1] = make_float4(t[2].in_block.x, t[2].in_block.y, t[3].in_block.x, t[3].in_block.y);
  *reinterpret_cast<float4*>(tab->col + 4 * lane) = make_float4(t[0].col, t[1].col, t[2].col, t[3].col);
  *reinterpret_cast<float4*>(tab->c1 + 4 * lane) = make_float4(t[0].c1, t[1].c1, t[2].c1, t[3].c1);
  *reinterpret_cast<float4*>(tab->weight + 4 * lane) = make_float4(t[0].weight, t[1].weight, t[2].weight, t[3].weight);
  store_whole(tab, g, lane);
}

// Products over operands in 128-row tiles; the descriptor of the first k-step is made once and the others
// are sums with constants (made anew each they took the issuing thread 125 cycles an instruction, twice what
// it takes to run).  N = 64: the second block is not there, or its rows of the result are not used.
template <int K> __device__ __forceinline__ void mma_kk_body(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add) {  // both K-major
  const uint64_t da = desc_k(a, 0), db = desc_k(b, 0);
#pragma unroll
  for (int kk = 0; kk < K / 16; ++kk)
    umma_bf16(d, da + step_of<kAlong>(kk), db + step_of<kAlong>(kk), id, (add || kk > 0) ? 1u : 0u);
}
__device__ __forceinline__ void mma_mm_body(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add) {  // K down the rows of both
  const uint64_t da = desc_mn(a, 0), db = desc_mn(b, 0);
#pragma unroll
  for (int kk = 0; kk < kC / 16; ++kk)
    umma_bf16(d, da + step_of<kDown>(kk), db + step_of<kDown>(kk), id, (add || kk > 0) ? 1u : 0u);
}
__device__ __forceinline__ void mma_tm_body(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t id) {  // A in tensor memory
  const uint64_t db = desc_mn(b, 0);
#pragma unroll
  for (int kk = 0; kk < kC / 16; ++kk) umma_bf16_ta(d, a_tmem + kk * 8, db + step_of<kDown>(kk), id, kk > 0 ? 1u : 0u);
}
// SHORT: as calls (see run_job on the length of the code)
template <int K> static __device__ __noinline__ void mma_kk_call(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add) {
  mma_kk_body<K>(d, a, b, id, add);
}
static __device__ __noinline__ void mma_mm_call(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add) { mma_mm_body(d, a, b, id, add); }
static __device__ __noinline__ void mma_tm_call(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t id) { mma_tm_body(d, a_tmem, b, id); }
template <bool SHORT, int K> __device__ __forceinline__ void mma_kk(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add) {
  if (SHORT) mma_kk_call<K>(d, a, b, id, add);
  else mma_kk_body<K>(d, a, b, id, add);
}
template <bool SHORT> __device__ __forceinline__ void mma_mm(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool add) {
  if (SHORT) mma_mm_call(d, a, b, id, add);
  else mma_mm_body(d, a, b, id, add);
}
template <bool SHORT> __device__ __forceinline__ void mma_tm(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t id) {
  if (SHORT) mma_tm_call(d, a_tmem, b, id);
  else mma_tm_body(d, a_tmem, b, id);
}

// ---- pairs of floats
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(f2 a) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(a));
  return v;
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
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack2(f2 a) {
  const float2 v = unpair(a);
  return pack_bf16x2(v.x, v.y);
}
__device__ __forceinline__ f2 unpack2(uint32_t u) { return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)); }
// x as bf16; what that leaves of it stays in x
__device__ __forceinline__ uint32_t take2(f2& x) {
  const uint32_t h = pack2(x);
  x = fma2(unpack2(h), pair(-1.f, -1.f), x);
  return h;
}
// tensor memory columns
// (the masked scores, 16 bits, take the middle of the scores' place: each half of a row's columns falls within
// its own, and is written behind what has been read)
constexpr uint32_t kTmP = 0, kTmPb = 32, kTmO1 = 128, kTmO2 = 256, kTmM = 384;

// Rows from n on of a tile, which belong to other sequences: zeros, whatever they hold.
static __device__ __noinline__ void zero_rows(unsigned char* tile, uint32_t full, uint32_t par, int i, int n, int c0, int pieces,
                                              unsigned* err) {
  wait_at(full, par, err);
  if (i >= n)
    for (int c = c0; c < c0 + pieces; ++c) *reinterpret_cast<uint4*>(tile + swz16(i, c)) = make_uint4(0u, 0u, 0u, 0u);
}

// One segment of one head.  DX: columns of q and k, DY of v (and w) and of the output.
//   NT = 4: w is loaded too, the state has three parts, row products are written.
// Tiles go through a ring of buffers in the order of use.  Of the buffers that are left one
// holds the state and another its low part (the least part goes first, in the high one's place), and once
// q M^T is done that of k' (k' high takes k's place).  The third part of k' takes the state's place (NT = 4) or, where q M^T waits for the outputs' way out and k' would wait
// for it, one of the ring's (`third`: a state that is returned; 16384 tokens, 16 heads: 65 us where 58 with two parts).
// The output is staged in v's place, with NT = 4 in w's.  The roles' code is kept short, in loops: unrolled
// (90 KB) it left the instruction cache and every phase waited for its instructions.  With NT = 4 it has to be
// shorter still, products and waits as calls (SHORT: 155 us where 190 with two parts, 63 % of requests hit instead of 52; without
// them the forward takes 57 us where 69).  What a chunk adds
// to the state is summed by itself in tensor memory and added to the state in registers: the tensor
// cores' sums round towards zero, which over the chunks of a long memory adds up (6e-6 of a state
// at 16384 tokens).  The chain from chunk to chunk is this addition alone.
//
// Only the state on entry comes from the kernels before: everything else starts without them.
template <int DX, int DY, int NT, bool REV, bool SHORT>
__device__ __forceinline__ void run_job(const TcParams& p, const TcJob& job, const CUtensorMap* mq, const CUtensorMap* mk,
                                        const CUtensorMap* mv, const CUtensorMap* mw, const CUtensorMap* mo, bool q_key,
                                        bool k_key, bool v_key, bool w_key, bool trans, const LaSegment& sg, int slot, int h,
                                        unsigned char* s) {
  constexpr bool LO = NT == 4;
  const bool third = !LO && job.last;
  const int ring = third ? kBufs - 3 : kBufs - 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = h / (p.seqs.H / p.seqs.Hk);
  const size_t row = ((size_t)sg.row_b * p.seqs.H + h) * p.seqs.T + sg.start;
  const size_t krow = ((size_t)sg.row_b * p.seqs.Hk + hk) * p.seqs.T + sg.start;
  const int chunks = (sg.n + kC - 1) / kC;
  const int elems = DX * DY;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s + Sm::kBars);
  const uint32_t sbars = smem_u32(bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + Sm::kSlot);
  Tab* tab = reinterpret_cast<Tab*>(s + Sm::kLog);
  unsigned char* mb = s + (kBufs - 2) * kTile;
  unsigned char* mlo = mb + kTile;
  auto chunk_at = [&](int x) { return REV ? chunks - 1 - x : x; };
  // where in the ring a chunk's tiles begin, and on which time round; tile j's buffer, the parity of its arrival
  int rb = 0, rn = 0;
  auto next_chunk = [&]() {
    rb += NT;
    if (rb >= ring) {
      rb -= ring;
      ++rn;
    }
  };
  auto buf = [&](int j) { return rb + j >= ring ? rb + j - ring : rb + j; };
  auto par = [&](int j) { return (rb + j >= ring ? rn + 1 : rn) & 1; };
  auto wait = [&](int b, uint32_t parity) {
    if (SHORT || !try_wait_at(sbars + 8 * b, parity)) wait_at(sbars + 8 * b, parity, p.err);
  };
  constexpr int Q = 0, K = 1, V = 2, W = 3, OUT = LO ? W : V;

  if (tid == 0) {
    for (int b = 0; b < kNumBars; ++b)
      mbar_init(bars + b, b == kMb || b == kMhi || b == kKp ? kStateThreads : b == kP || b == kRead || b == kStaged ? kRowThreads : b == kTab ? 32 : 1);
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sbuf = smem_u32(s);

  if (warp == kIssueWarp + 1) {
    if (lane == 0) {
#pragma unroll 1
      for (int x = 0; x < chunks; ++x, next_chunk()) {
        const int t0 = chunk_at(x) * kC;
#pragma unroll 1
        for (int j = 0; j < NT; ++j) {
          const int b = buf(j), n = rb + j >= ring ? rn + 1 : rn;
          if (n > 0) wait(kEmpty + b, (n - 1) & 1);
          const CUtensorMap* m = j == W ? mw : j == Q ? mq : j == K ? mk : mv;
          const bool key = j == W ? w_key : j == Q ? q_key : j == K ? k_key : v_key;
          const int cols = j == W || j == V ? DY : DX;
          const int r = (int)((key ? krow : row) + t0);
          uint64_t* bar = bars + kFull + b;
          mbar_arrive_expect_tx(bar, (uint32_t)(cols / 64) * kHalf);
          for (int c = 0; c < cols / 64; ++c) tma_load_2d(s + b * kTile + c * kHalf, m, bar, 64 * c, r);
        }
      }
    }
  } else if (warp == kIssueWarp) {
    if (lane == 0) {
      const uint32_t smb = sbuf + (kBufs - 2) * kTile, low = smb + kTile, rest = LO ? smb : smb - kTile;
#pragma unroll 1
      for (int x = 0; x < chunks; ++x, next_chunk()) {
        const int ph = x & 1;
        const uint32_t q = sbuf + buf(Q) * kTile, k = sbuf + buf(K) * kTile, v = sbuf + buf(V) * kTile;
        wait(kFull + buf(Q), par(Q));
        wait(kFull + buf(K), par(K));
        tc_fence_after();
        mma_kk<SHORT, DX>(tmem + kTmP, q, k, idesc_bf16(128, kC, false, false), false);
        if (LO) {
          if (x > 0) wait(kRead, (x - 1) & 1);  // the last outputs have been read
          wait(kFull + buf(W), par(W));
          wait(kFull + buf(V), par(V));
          tc_fence_after();
          mma_kk<SHORT, DY>(tmem + kTmO2, sbuf + buf(W) * kTile, v, idesc_bf16(128, kC, false, false), false);
        }
        umma_commit(bars + kS1);
        wait(kMb, ph);
        if (!LO && x > 0) wait(kRead, (x - 1) & 1);
        tc_fence_after();
        mma_kk<SHORT, DX>(tmem + kTmO1, q, smb, idesc_bf16(128, DY, false, false), false);
        if (LO) {  // the least part was in the high one's place
          umma_commit(bars + kLeast);
          mma_kk<SHORT, DX>(tmem + kTmO1, q, low, idesc_bf16(128, DY, false, false), true);
          wait(kMhi, ph);
          tc_fence_after();
          mma_kk<SHORT, DX>(tmem + kTmO1, q, smb, idesc_bf16(128, DY, false, false), true);
        }
        umma_commit(bars + kS2);
        umma_commit(bars + kEmpty + buf(Q));
        auto output = [&]() {
          wait(kP, ph);
          tc_fence_after();
          mma_tm<SHORT>(tmem + kTmO2, tmem + kTmPb, v, idesc_bf16(128, DY, false, true));
          umma_commit(bars + kS3);
        };
        if (LO) output();
        wait(kKp, ph);
        if (!LO) wait(kFull + buf(V), par(V));
        tc_fence_after();
        // the least first: a sum is cut off as often as it is added to, and only large ones by much
        mma_mm<SHORT>(tmem + kTmM, v, low, idesc_bf16(128, DX, true, true), false);
        if (LO || third) mma_mm<SHORT>(tmem + kTmM, v, rest, idesc_bf16(128, DX, true, true), true);
        mma_mm<SHORT>(tmem + kTmM, v, k, idesc_bf16(128, DX, true, true), true);
        umma_commit(bars + kS4);
        umma_commit(bars + kEmpty + buf(K));
        if (LO) umma_commit(bars + kEmpty + buf(V));
        if (!LO) output();
      }
    }
  } else if (warp == kIssueWarp + 2) {
    if (lane == 0) {
#pragma unroll 1
      for (int x = 0; x < chunks; ++x, next_chunk()) {
        const int t0 = chunk_at(x) * kC;
        wait(kStaged, x & 1);
        if (!job.out_f32 && sg.n - t0 >= kC) {
          for (int c = 0; c < DY / 64; ++c) tma_store_2d(mo, s + buf(OUT) * kTile + c * kHalf, 64 * c, (int)(row + t0));
          bulk_commit();
          bulk_wait_read0();
        }
        mbar_arrive(bars + kStored);
        mbar_arrive(bars + kEmpty + buf(OUT));
      }
      bulk_wait0();
    }
  } else if (warp == kIssueWarp + 3) {
    const float* la = p.log_alpha + (p.per_head ? (size_t)h : row);
    float next[4];
    auto load = [&](int x) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = chunk_at(x) * kC + 4 * lane + e;
        next[e] = t < sg.n ? la_log(la[p.per_head ? 0 : t]) : 0.f;
      }
    };
    load(0);
#pragma unroll 1
    for (int x = 0; x < chunks; ++x) {
      const ChunkLog g = chunk_log(next, lane);
      const int n = min(kC, sg.n - chunk_at(x) * kC);
      TabEntry t[4];
      if (!SHORT)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = make_entry<REV>(g, g.past[e], 4 * lane + e < n, p.scale);
      if (x + 1 < chunks) load(x + 1);
      if (x > 0) {  // the groups are done with the last chunk's
        wait(kP, (x - 1) & 1);
        wait(kKp, (x - 1) & 1);
      }
      if (SHORT) store_short<REV>(tab, g, lane, n, p.scale);
      else store_tab(tab, t, g, lane);
      mbar_arrive(bars + kTab);
    }
  } else if (warp >= kStateWarp) {
    // ---- the state: row i (of DY), a part of its columns; then k': token i, a part of the columns
    constexpr int N = DX / (kStateThreads / kC), kVN = DY / 8 / (kStateThreads / kC);
    const int w4 = warp & 3, part = (warp - kStateWarp) >> 2, i = 32 * w4 + lane;
    const uint32_t tm = tmem + kTmM + ((uint32_t)(32 * w4) << 16) + part * N;
    f2 M[N / 2];
    wait_for_previous();
    {
      const float* in = job.in ? job.in + ((size_t)(job.in_by_slot ? slot : sg.seq) * p.seqs.H + h) * elems : nullptr;
#pragma unroll
      for (int e = 0; e < N / 2; ++e) M[e] = 0ull;
      if (in && i < DY) {
        if (trans) {  // lies [DX][DY]
#pragma unroll
          for (int e = 0; e < N / 2; ++e)
            M[e] = pair(in[(size_t)(part * N + 2 * e) * DY + i], in[(size_t)(part * N + 2 * e + 1) * DY + i]);
        } else {
#pragma unroll
          for (int e = 0; e < N / 2; e += 2) {
            const float4 v = *reinterpret_cast<const float4*>(in + (size_t)i * DX + part * N + 2 * e);
            M[e] = pair(v.x, v.y);
            M[e + 1] = pair(v.z, v.w);
          }
        }
      }
    }
    float2 d = make_float2(0.f, 1.f);  // of the chunk before
#pragma unroll 1
    for (int x = 0;; ++x, next_chunk()) {
      const int ph = x & 1, t0 = chunk_at(x) * kC, n = min(kC, sg.n - t0);
      if (x > 0) {  // M <- decay M + what the chunk before added; near 1 the decay as M + expm1 M (la.cuh)
        LL_GROUP_WAIT(warp == kStateWarp, kBarState, kStateThreads, wait(kS4, (x - 1) & 1));
        tc_fence_after();
        const f2 df = pair(d.x, d.x);
        const bool near = d.y != 0.f;
#pragma unroll
        for (int c = 0; c < N; c += 16) {
          float y[16];
          tmem_ld16(tm + c, y);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f2& m = M[(c >> 1) + e];
            const f2 yy = pair(y[2 * e], y[2 * e + 1]);
            m = fma2(m, df, near ? add2(m, yy) : yy);
          }
        }
      }
      if (x == chunks) break;
      auto put_state = [&](bool least) {  // (NT = 4) the two lower parts, then the high one in the least one's place
        if (DY == 128 || w4 < 2) {
#pragma unroll
          for (int c = 0; c < N; c += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              f2 a = M[(c >> 1) + v];
              hi[v] = LO && least ? take2(a) : pack2(a);
              if (LO && least) {
                lo[v] = take2(a);
                hi[v] = pack2(a);
              }
            }
            const uint32_t at = swz16(i, (part * N + c) >> 3);
            *reinterpret_cast<uint4*>(mb + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (LO && least) *reinterpret_cast<uint4*>(mlo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async_shared();
      };
      put_state(true);
      tc_fence_before();
      mbar_arrive(bars + kMb);
      if (LO) {
        LL_GROUP_WAIT(warp == kStateWarp, kBarState, kStateThreads, wait(kLeast, ph));
        put_state(false);
        mbar_arrive(bars + kMhi);
      }
      // k' high in k's place, low in that of the state's low part
      unsigned char* kb = s + buf(K) * kTile;
      LL_GROUP_WAIT(warp == kStateWarp, kBarState, kStateThreads, {
        wait(kTab, ph);
        wait((LO ? kS2 : kS1), ph);
        wait(kFull + buf(K), par(K));  // (long complete: the copy's writes, seen from here)
      });
      const float weight = tab->weight[i];
      d = tab->decay;
      const f2 ww = pair(weight, weight);
      const ptrdiff_t to_low = mlo - kb;
      const int low_to_rest = LO ? kTile : 2 * kTile;  // downwards
#pragma unroll 1
      for (int e8 = 0; e8 < N / 8; e8 += 2) {  // two pieces at a time: their chains run side by side
        uint4 v[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) v[g] = *reinterpret_cast<const uint4*>(kb + swz16(i, part * (N / 8) + e8 + g));
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          unsigned char* at = kb + swz16(i, part * (N / 8) + e8 + g);
          uint32_t hi[4] = {v[g].x, v[g].y, v[g].z, v[g].w}, lo[4], rest[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f2 a = mul2(unpack2(hi[e]), ww);
            hi[e] = take2(a);
            lo[e] = take2(a);
            rest[e] = pack2(a);
          }
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(at + to_low) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          if (LO || third) *reinterpret_cast<uint4*>(at + to_low - low_to_rest) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
        }
      }
      if (n < kC) {  // rows of other sequences: zeros, whatever they hold
        zero_rows(kb, sbars + 8 * (kFull + buf(K)), par(K), i, n, part * (N / 8), N / 8, p.err);
        zero_rows(mlo, sbars + 8 * (kFull + buf(K)), par(K), i, n, part * (N / 8), N / 8, p.err);
        if (LO || third) zero_rows(mlo - low_to_rest, sbars + 8 * (kFull + buf(K)), par(K), i, n, part * (N / 8), N / 8, p.err);
      }
      if (!LO && n < kC) zero_rows(s + buf(V) * kTile, sbars + 8 * (kFull + buf(V)), par(V), i, n, part * kVN, kVN, p.err);
      fence_proxy_async_shared();
      mbar_arrive(bars + kKp);
    }
    if (job.last && (REV ? sg.num == 0 : (long long)sg.num * p.seg + sg.n == sg.seq_len)) {
      float* dst = job.last + ((size_t)sg.seq * p.seqs.H + h) * elems;
      if (i < DY) {
        if (trans) {  // lies [DX][DY]
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            const float2 a = unpair(M[e]);
            dst[(size_t)(part * N + 2 * e) * DY + i] = a.x;
            dst[(size_t)(part * N + 2 * e + 1) * DY + i] = a.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < N / 2; e += 2) {
            const float2 a = unpair(M[e]), b = unpair(M[e + 1]);
            *reinterpret_cast<float4*>(dst + (size_t)i * DX + part * N + 2 * e) = make_float4(a.x, a.y, b.x, b.y);
          }
        }
      }
    }
    tc_fence_before();
  } else {
    // ---- scores and outputs: token i, half of the columns
    constexpr int N = DY / 2;
    const int w4 = warp & 3, half = warp >> 2, i = 32 * w4 + lane;
    const uint32_t lanes = (uint32_t)(32 * w4) << 16;
#pragma unroll 1
    for (int x = 0; x < chunks; ++x, next_chunk()) {
      const int ph = x & 1, t0 = chunk_at(x) * kC, n = min(kC, sg.n - t0);
      LL_GROUP_WAIT(warp == 0, kBarRows, kRowThreads, {
        wait(kTab, ph);
        wait(kS1, ph);
      });
      tc_fence_after();
      const float2 own_log = tab->in_block[i];
      // to the border of the row's block, and over the blocks that can lie between
      const float2 bw = tab->blk[w4], b1 = tab->blk[1], b2 = tab->blk[2];
      const float own = REV ? (bw.x - own_log.x) + (bw.y - own_log.y) : own_log.x;
      const f2 own2 = pair(own_log.x, own_log.y);
      const float c1 = tab->c1[i], c2 = p.scale;  // (the scores take the scale with them)
      float rs = 0.f;
#pragma unroll 1
      for (int jj = 0; jj < 4; ++jj) {  // 16 columns at a time
        const int j0 = half ? 64 + 16 * jj : 48 - 16 * jj, J = j0 >> 5;
        uint32_t pk[8];
        if (REV ? J < w4 : J > w4) {
#pragma unroll
          for (int e = 0; e < 8; ++e) pk[e] = 0u;
        } else {
          float y[16];
          f2 dec[8];
          tmem_ld16(tmem + kTmP + lanes + j0, y);
          if (J == w4) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(tab->in_block + j0 + e);
              const f2 minus = pair(-1.f, -1.f);
              const float2 d0 = unpair(REV ? fma2(own2, minus, l.x) : fma2(l.x, minus, own2));
              const float2 d1 = unpair(REV ? fma2(own2, minus, l.y) : fma2(l.y, minus, own2));
              dec[e / 2] = pair(c2 * ex2(d0.x + d0.y), c2 * ex2(d1.x + d1.y));
            }
          } else {
            float between = own;
            if (REV ? 1 > w4 && 1 < J : 1 < w4 && 1 > J) between += b1.x;
            if (REV ? 2 > w4 && 2 < J : 2 < w4 && 2 > J) between += b2.x;
            const float f = c2 * ex2(between);
            const f2 ff = pair(f, f);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(tab->col + j0 + e);
              dec[e / 2] = mul2(c.x, ff);
              dec[e / 2 + 1] = mul2(c.y, ff);
            }
          }
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 v = unpair(mul2(pair(y[2 * e], y[2 * e + 1]), dec[e]));
            y[2 * e] = v.x;
            y[2 * e + 1] = v.y;
          }
          // columns [from, to) of these are in the mask; of the others nothing, whatever they hold
          const bool edge = J == w4 || n < kC;
          const int from = REV ? i - j0 : 0, to = REV ? n - j0 : min(i + 1, n) - j0;
          if (edge) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if ((REV && e < from) || e >= to) y[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) pk[e] = pack_bf16x2(y[2 * e], y[2 * e + 1]);
          if (LO) {
            float w[16];
            tmem_ld16(tmem + kTmO2 + lanes + j0, w);
            tmem_ld_wait();
            if (edge) {  // (a row's own pair is left out)
              const int end = REV ? to : min(i, n) - j0;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if ((REV && e <= from) || e >= end) w[e] = 0.f;
            }
            f2 a0 = 0ull, a1 = 0ull;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              a0 = fma2(pair(y[2 * e], y[2 * e + 1]), pair(w[2 * e], w[2 * e + 1]), a0);
              a1 = fma2(pair(y[2 * e + 2], y[2 * e + 3]), pair(w[2 * e + 2], w[2 * e + 3]), a1);
            }
            const float2 a = unpair(add2(a0, a1));
            rs += a.x + a.y;
          }
        }
        tmem_st8(tmem + kTmPb + lanes + (j0 >> 1), pk);
      }
      tmem_st_wait();
      tc_fence_before();
      if (LO && n < kC) zero_rows(s + buf(V) * kTile, sbars + 8 * (kFull + buf(V)), par(V), i, n, half * (DY / 16), DY / 16, p.err);
      if (LO && n < kC) fence_proxy_async_shared();
      mbar_arrive(bars + kP);
      LL_GROUP_WAIT(warp == 0, kBarRows, kRowThreads, {
        wait(kS3, ph);
        if (LO) wait(kFull + buf(W), par(W));
        if (x > 0) wait(kStored, (x - 1) & 1);  // (the stores never fall two chunks behind)
      });
      tc_fence_after();
      f2 dot = 0ull;
      float* of = job.out_f32 ? job.out_f32 + (row + t0 + i) * DY + half * N : nullptr;
      unsigned char* stage = s + buf(OUT) * kTile;
      const f2 k1 = pair(c1, c1);
#pragma unroll 1
      for (int c = 0; c < N; c += 16) {
        float a[16], b[16];
        tmem_ld16(tmem + kTmO1 + lanes + half * N + c, a);
        tmem_ld16(tmem + kTmO2 + lanes + half * N + c, b);
        tmem_ld_wait();
        uint4* at[2] = {reinterpret_cast<uint4*>(stage + swz16(i, (half * N + c) >> 3)),
                        reinterpret_cast<uint4*>(stage + swz16(i, ((half * N + c) >> 3) + 1))};
        if (LO) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint4 v = *at[g];
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              dot = fma2(pair(a[8 * g + 2 * e], a[8 * g + 2 * e + 1]), unpack2(u[e]), dot);
            }
          }
        }
        f2 y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fma2(pair(a[2 * e], a[2 * e + 1]), k1, pair(b[2 * e], b[2 * e + 1]));
        if (of) {
          if (i < n)
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 v0 = unpair(y[e]), v1 = unpair(y[e + 1]);
              *reinterpret_cast<float4*>(of + c + 2 * e) = make_float4(v0.x, v0.y, v1.x, v1.y);
            }
        } else {
#pragma unroll
          for (int g = 0; g < 2; ++g)
            *at[g] = make_uint4(pack2(y[4 * g]), pack2(y[4 * g + 1]), pack2(y[4 * g + 2]), pack2(y[4 * g + 3]));
        }
      }
      tc_fence_before();
      mbar_arrive(bars + kRead);
      if (LO && i < n) job.part[half * p.part_stride + row + t0 + i] = fmaf(c1, unpair(dot).x + unpair(dot).y, rs);
      if (!of && n < kC) {
        named_bar_sync(kBarRows, kRowThreads);
        store_rows(static_cast<char*>(job.out) + (row + t0) * DY * 2, stage, n, DY, tid, kRowThreads);
      }
      fence_proxy_async_shared();
      mbar_arrive(bars + kStaged);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Nothing but a state: the sequence is empty.
__device__ __forceinline__ void copy_state(const TcParams& p, const TcJob& job, const LaSegment& sg, int slot, int h) {
  wait_for_previous();
  if (!job.last) return;
  const int elems = p.dk * p.dv;
  float* dst = job.last + ((size_t)sg.seq * p.seqs.H + h) * elems;
  const float* in = job.in ? job.in + ((size_t)(job.in_by_slot ? slot : sg.seq) * p.seqs.H + h) * elems : nullptr;
  for (int e = threadIdx.x; e < elems; e += kThreads) dst[e] = in ? in[e] : 0.f;
}
__device__ __forceinline__ bool enter(const TcParams& p, int item, LaSegment& sg, int& slot, int& h, const unsigned char* s) {
  let_next_launch();
  if (smem_u32(s) & 1023u) {
    if (threadIdx.x == 0) raise_error(p.err, kErrDeviceArg);
    return false;
  }
  if (item == 0 && p.seqs.starts)  // every sequence's bounds, whoever finds it
    for (int i = threadIdx.x; i < p.seqs.n; i += kThreads) {
      GdrSeq q;
      if (!gdr_seq(p.seqs, i, q)) raise_error(p.err, kErrDeviceArg);
    }
  h = item % p.seqs.H;
  slot = item / p.seqs.H;
  if (la_find(p.seqs, slot, p.seg, sg, p.err)) return true;
  wait_for_previous();  // (what follows this launch takes those before it as ended)
  return false;
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) la_tc_fwd_kernel(const __grid_constant__ FwdMaps m, const __grid_constant__ TcParams p) {
  extern __shared__ __align__(1024) unsigned char s[];
  LaSegment sg;
  int slot, h;
  if (!enter(p, blockIdx.x, sg, slot, h, s)) return;
  if (sg.n == 0) return copy_state(p, p.job[0], sg, slot, h);
  run_job<DK, DV, 3, false, false>(p, p.job[0], &m.q, &m.k, &m.v, nullptr, &m.o, true, true, false, false, false, sg, slot, h, s);
}

// dq, dv, dk of one segment and head side by side: they read the same tiles
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) la_tc_bwd_kernel(const __grid_constant__ BwdMaps m, const __grid_constant__ TcParams p) {
  extern __shared__ __align__(1024) unsigned char s[];
  LaSegment sg;
  int slot, h;
  const int item = blockIdx.x / 3, what = blockIdx.x - 3 * item;
  if (!enter(p, item, sg, slot, h, s)) return;
  if (sg.n == 0) {
    if (what == 1) copy_state(p, p.job[1], sg, slot, h);
    return;
  }
  if (what == 0) run_job<DV, DK, 4, false, true>(p, p.job[0], &m.dout, &m.v, &m.k, &m.q, &m.dq, false, false, true, true, true, sg, slot, h, s);
  else if (what == 1) run_job<DK, DV, 4, true, true>(p, p.job[1], &m.k, &m.q, &m.dout, &m.v, &m.dv, true, true, false, false, false, sg, slot, h, s);
  else run_job<DV, DK, 3, true, true>(p, p.job[2], &m.v, &m.dout, &m.q, nullptr, &m.dk, false, false, true, false, true, sg, slot, h, s);
}

// ---------------------------------------------------------------- sums of the segments
// What a segment adds to the state behind it (DIR 0: K, V, chunks from the last on)
// or to its gradient before it (DIR 1: Q, dO, from the first on), with the weights
// taken to the segment's border.  A chunk's two products go to one of two accumulators in
// tensor memory and from there are added up in registers (see above), beside the next
// chunk's.  Four threads to a row.
constexpr int kSumGroup = 512;
constexpr int kSumThreads = kSumGroup + 128;  // products in warp 16, copies in 17, weights in 18
struct SumParams {
  GdrSeqs seqs;
  int seg, per_head, dk, dv, dirs;
  float scale;
  const float* log_alpha;
  float* sums[2];
  float* log_decay;
  unsigned* err;
};
struct SumMaps {
  CUtensorMap k, v, q, dout;
};
template <int DK, int DV, int PARTS>  // of k'
__global__ void __launch_bounds__(kSumThreads, 1) la_tc_sum_kernel(const __grid_constant__ SumMaps m, const __grid_constant__ SumParams p) {
  extern __shared__ __align__(1024) unsigned char s[];
  let_next_launch();
  if (smem_u32(s) & 1023u) {
    if (threadIdx.x == 0) raise_error(p.err, kErrDeviceArg);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = blockIdx.x / p.dirs, dir = blockIdx.x - item * p.dirs;
  const int h = item % p.seqs.H, slot = item / p.seqs.H, hk = h / (p.seqs.H / p.seqs.Hk);
  LaSegment sg;
  if (!la_find(p.seqs, slot, p.seg, sg, p.err)) return;
  const size_t row = ((size_t)sg.row_b * p.seqs.H + h) * p.seqs.T + sg.start;
  const size_t krow = ((size_t)sg.row_b * p.seqs.Hk + hk) * p.seqs.T + sg.start;
  const float* la = p.log_alpha + (p.per_head ? (size_t)h : row);
  const bool edge = dir ? sg.num == 0 : (long long)sg.num * p.seg + sg.n == sg.seq_len;
  const bool work = sg.n > 0 && !edge;  // (nothing needs the last (first) segment's sum)
  const int chunks = work ? (sg.n + kC - 1) / kC : 0;
  float* dst = p.sums[dir] + ((size_t)slot * p.seqs.H + h) * (DK * DV);
  if (!work) {  // (its log decay is wanted all the same, of the first segment backwards by DIR 0)
    if (dir == 0 && warp == 0) {
      float g = 0.f;
      for (int t = lane; t < sg.n; t += 32) g += la_log(la[p.per_head ? 0 : t]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) g += __shfl_xor_sync(0xffffffffu, g, o);
      if (lane == 0) p.log_decay[(size_t)slot * p.seqs.H + h] = g;
    }
    if (sg.n == 0)
      for (int e = tid; e < DK * DV; e += kSumThreads) dst[e] = 0.f;
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(s + Sm::kBars);  // full, empty, k' ready, products done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + Sm::kSlot);
  constexpr int kSumRing = PARTS == 2 ? 6 : 4;  // buffers of tiles; those behind them hold the lower parts
  constexpr int kReady = 2 * kSumRing, kDone = kReady + 1, kWeights = kDone + 1;
  float* weights = reinterpret_cast<float*>(s + Sm::kLog);  // of a chunk's rows
  if (tid == 0) {
    for (int b = 0; b <= kWeights; ++b) mbar_init(bars + b, b == kReady ? kSumGroup : b == kWeights ? 32 : 1);
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, sbuf = smem_u32(s);
  unsigned char* low = s + kSumRing * kTile;
  auto chunk_at = [&](int x) { return dir ? x : chunks - 1 - x; };

  if (warp == 17) {
    if (lane == 0) {
      for (int x = 0, i = 0; x < chunks; ++x)
        for (int j = 0; j < 2; ++j, ++i) {
          const int b = i % kSumRing, n = i / kSumRing;
          if (n > 0) wait_bar(bars + kSumRing + b, (n - 1) & 1, p.err);
          const CUtensorMap* map = j == 0 ? (dir ? &m.q : &m.k) : (dir ? &m.dout : &m.v);
          const int cols = j == 0 ? DK : DV, r = (int)((j == 0 ? krow : row) + chunk_at(x) * kC);
          mbar_arrive_expect_tx(bars + b, (uint32_t)(cols / 64) * kHalf);
          for (int c = 0; c < cols / 64; ++c) tma_load_2d(s + b * kTile + c * kHalf, map, bars + b, 64 * c, r);
        }
    }
  } else if (warp == 16) {
    if (lane == 0) {
      for (int x = 0; x < chunks; ++x) {
        const int bk = 2 * x % kSumRing, bv = bk + 1, n = 2 * x / kSumRing;
        const uint32_t acc = tmem + (x & 1) * 128;
        wait_bar(bars + bv, n & 1, p.err);
        wait_bar(bars + kReady, x & 1, p.err);
        tc_fence_after();
        mma_mm<false>(acc, sbuf + bv * kTile, sbuf + kSumRing * kTile, idesc_bf16(128, DK, true, true), false);
        if (PARTS == 3) mma_mm<false>(acc, sbuf + bv * kTile, sbuf + (kSumRing + 1) * kTile, idesc_bf16(128, DK, true, true), true);
        mma_mm<false>(acc, sbuf + bv * kTile, sbuf + bk * kTile, idesc_bf16(128, DK, true, true), true);
        umma_commit(bars + kSumRing + bk);
        umma_commit(bars + kSumRing + bv);
        umma_commit(bars + kDone);
      }
    }
  } else if (warp == 18) {
    float next[4];
    auto load = [&](int x) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = chunk_at(x) * kC + 4 * lane + e;
        next[e] = t < sg.n ? la_log(la[p.per_head ? 0 : t]) : 0.f;
      }
    };
    long long run = 0;  // to the segment's border (cut off where its exponential is long zero or infinite)
    float bad = 0.f;
    load(0);
#pragma unroll 1
    for (int x = 0; x < chunks; ++x) {
      const ChunkLog g = chunk_log(next, lane);
      const int n = min(kC, sg.n - chunk_at(x) * kC);
      if (x + 1 < chunks) load(x + 1);
      bad += g.bad;
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = expf(log_float(run + (dir ? g.past[e] : g.total - g.past[e])) + bad) * (dir ? p.scale : 1.f);
        if (4 * lane + e >= n) w[e] = 0.f;
      }
      if (x > 0) wait_bar(bars + kReady, (x - 1) & 1, p.err);  // the rows have read the last chunk's
      *reinterpret_cast<float4*>(weights + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
      run = min(max(run + g.total, -((long long)1 << 60)), (long long)1 << 60);
      mbar_arrive(bars + kWeights);
    }
    if (dir == 0 && lane == 0) p.log_decay[(size_t)slot * p.seqs.H + h] = log_float(run) + bad;
  } else if (warp < 16) {
    constexpr int N = DK / 4;
    const int w4 = warp & 3, i = 32 * w4 + lane, part = warp >> 2;
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
    auto add = [&](int x) {  // chunk x's products, which are complete
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < N; c += 16) {
        float y[16];
        tmem_ld16(tmem + (x & 1) * 128 + ((uint32_t)(32 * w4) << 16) + part * N + c, y);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[c + e] += y[e];
      }
      tc_fence_before();
    };
    for (int x = 0; x < chunks; ++x) {
      const int b = 2 * x % kSumRing, n = min(kC, sg.n - chunk_at(x) * kC);
      LL_GROUP_WAIT(warp == 0, kBarRows, kSumGroup, {
        wait_bar(bars + kWeights, x & 1, p.err);
        wait_bar(bars + b, 2 * x / kSumRing & 1, p.err);
      });
      const float weight = weights[i];
      unsigned char* kb = s + b * kTile;
      uint32_t lo[N / 2], rest[PARTS == 3 ? N / 2 : 1];
      const f2 ww = pair(weight, weight);
#pragma unroll
      for (int e8 = 0; e8 < N / 8; ++e8) {
        uint4* at = reinterpret_cast<uint4*>(kb + swz16(i, part * (N / 8) + e8));
        const uint4 v = *at;
        uint32_t hi[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f2 y = mul2(unpack2(hi[e]), ww);
          hi[e] = take2(y);
          lo[4 * e8 + e] = PARTS == 3 ? take2(y) : pack2(y);
          if (i >= n) hi[e] = lo[4 * e8 + e] = 0u;
          if (PARTS == 3) rest[4 * e8 + e] = i >= n ? 0u : pack2(y);
        }
        *at = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      }
      if (n < kC) {  // rows of v behind the segment
        wait_bar(bars + b + 1, 2 * x / kSumRing & 1, p.err);
        if (i >= n)
#pragma unroll
          for (int e8 = 0; e8 < DV / 32; ++e8)
            *reinterpret_cast<uint4*>(kb + kTile + swz16(i, part * (DV / 32) + e8)) = make_uint4(0u, 0u, 0u, 0u);
      }
      if (x > 0) LL_GROUP_WAIT(warp == 0, kBarState, kSumGroup, wait_bar(bars + kDone, (x - 1) & 1, p.err));  // the low part's tile is free
#pragma unroll
      for (int e8 = 0; e8 < N / 8; ++e8) {
        unsigned char* at = low + swz16(i, part * (N / 8) + e8);
        *reinterpret_cast<uint4*>(at) = make_uint4(lo[4 * e8], lo[4 * e8 + 1], lo[4 * e8 + 2], lo[4 * e8 + 3]);
        if (PARTS == 3)
          *reinterpret_cast<uint4*>(at + kTile) = make_uint4(rest[4 * e8], rest[4 * e8 + 1], rest[4 * e8 + 2], rest[4 * e8 + 3]);
      }
      fence_proxy_async_shared();
      mbar_arrive(bars + kReady);
      if (x > 0) add(x - 1);
    }
    wait_bar(bars + kDone, (chunks - 1) & 1, p.err);
    add(chunks - 1);
    if (i < DV)
#pragma unroll
      for (int e = 0; e < N; e += 4)
        *reinterpret_cast<float4*>(dst + (size_t)i * DK + part * N + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
  }
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  auto f = fn.load(std::memory_order_acquire);
  if (!f) {  // (threads may look it up at once)
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &qr) != cudaSuccess ||
        qr != cudaDriverEntryPointSuccess)
      return nullptr;
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    fn.store(f, std::memory_order_release);
  }
  return f;
}
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)kC};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
TcParams tc_params(const LaArgs& a, int seg) {
  TcParams p{};
  p.seqs = la_seqs(a);
  p.seg = seg;
  p.per_head = a.per_head;
  p.dk = a.dk;
  p.dv = a.dv;
  p.scale = a.scale;
  p.part_stride = (size_t)a.B * a.H * a.T;
  p.log_alpha = a.log_alpha;
  p.err = a.err;
  return p;
}

}  // namespace

// bf16 io, head sizes of 64 and 128; rows are 32-bit coordinates of the copies
bool la_tc_formats(const LaArgs& a) {
  return a.io == LL_BF16 && a.dk >= 64 && a.dv >= 64 && (long long)a.B * a.H * a.T <= (1ll << 31) - 1 - kC;
}

ll_status la_tc_sum_launch(const LaArgs& a, int seg, size_t slots, int dirs, float* sum_s, float* sum_a, float* log_decay) {
  const uint64_t rows = (uint64_t)a.B * a.H * a.T, krows = (uint64_t)a.B * a.Hk * a.T;
  SumMaps m;
  if (!make_map(&m.k, a.k, krows, a.dk) || !make_map(&m.v, a.v, rows, a.dv) || !make_map(&m.q, a.q, krows, a.dk) ||
      !make_map(&m.dout, a.dout ? a.dout : a.v, rows, a.dv))
    return LL_ERR_CUDA;
  SumParams p{la_seqs(a), seg, a.per_head, a.dk, a.dv, dirs, a.scale, a.log_alpha, {sum_s, sum_a}, log_decay, a.err};
  const bool two = dirs == 1 && !a.state_out;  // (states that go no further than the outputs)
  auto kernel = two ? (a.dk == 128 ? (a.dv == 128 ? la_tc_sum_kernel<128, 128, 2> : la_tc_sum_kernel<128, 64, 2>)
                                   : (a.dv == 128 ? la_tc_sum_kernel<64, 128, 2> : la_tc_sum_kernel<64, 64, 2>))
                    : (a.dk == 128 ? (a.dv == 128 ? la_tc_sum_kernel<128, 128, 3> : la_tc_sum_kernel<128, 64, 3>)
                                   : (a.dv == 128 ? la_tc_sum_kernel<64, 128, 3> : la_tc_sum_kernel<64, 64, 3>));
  const size_t grid = slots * a.H * dirs;
  if (grid > 0x7fffffffull) return LL_ERR_UNSUPPORTED;
  return la_launch(false, kernel, dim3((unsigned)grid), kSumThreads, Sm::kBytes, a.stream, m, p);
}

ll_status la_tc_fwd_main(const LaArgs& a, int seg, size_t slots, const float* states, bool by_slot, bool after) {
  const uint64_t rows = (uint64_t)a.B * a.H * a.T, krows = (uint64_t)a.B * a.Hk * a.T;
  FwdMaps m;
  if (!make_map(&m.q, a.q, krows, a.dk) || !make_map(&m.k, a.k, krows, a.dk) || !make_map(&m.v, a.v, rows, a.dv) ||
      !make_map(&m.o, a.o, rows, a.dv))
    return LL_ERR_CUDA;
  TcParams p = tc_params(a, seg);
  p.job[0].in = states;
  p.job[0].in_by_slot = by_slot;
  p.job[0].last = a.state_out;
  p.job[0].out = a.o;
  auto kernel = a.dk == 128 ? (a.dv == 128 ? la_tc_fwd_kernel<128, 128> : la_tc_fwd_kernel<128, 64>)
                            : (a.dv == 128 ? la_tc_fwd_kernel<64, 128> : la_tc_fwd_kernel<64, 64>);
  const size_t grid = slots * a.H;
  if (grid > 0x7fffffffull) return LL_ERR_UNSUPPORTED;
  return la_launch(after, kernel, dim3((unsigned)grid), kThreads, Sm::kBytes, a.stream, m, p);
}

ll_status la_tc_bwd_main(const LaArgs& a, int seg, size_t slots, const float* states, const float* adjoints, bool by_slot, float* before,
                         float* ends, float* dq32, float* dk32, float* part_q, float* part_v, bool after) {
  const uint64_t rows = (uint64_t)a.B * a.H * a.T, krows = (uint64_t)a.B * a.Hk * a.T;
  BwdMaps m;
  if (!make_map(&m.q, a.q, krows, a.dk) || !make_map(&m.k, a.k, krows, a.dk) || !make_map(&m.v, a.v, rows, a.dv) ||
      !make_map(&m.dout, a.dout, rows, a.dv) || !make_map(&m.dq, a.dq, krows, a.dk) || !make_map(&m.dk, a.dkey, krows, a.dk) ||
      !make_map(&m.dv, a.dval, rows, a.dv))
    return LL_ERR_CUDA;
  TcParams p = tc_params(a, seg);
  p.job[0] = TcJob{states, ends, by_slot, dq32, part_q, a.dq};
  p.job[1] = TcJob{adjoints, before, by_slot, nullptr, part_v, a.dval};
  p.job[2] = TcJob{adjoints, nullptr, by_slot, dk32, nullptr, a.dkey};
  auto kernel = a.dk == 128 ? (a.dv == 128 ? la_tc_bwd_kernel<128, 128> : la_tc_bwd_kernel<128, 64>)
                            : (a.dv == 128 ? la_tc_bwd_kernel<64, 128> : la_tc_bwd_kernel<64, 64>);
  const size_t grid = slots * a.H * 3;
  if (grid > 0x7fffffffull) return LL_ERR_UNSUPPORTED;
  return la_launch(after, kernel, dim3((unsigned)grid), kThreads, Sm::kBytes, a.stream, m, p);
}

}  // namespace llattn

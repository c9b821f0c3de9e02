// The gated delta rule on the 5th-generation tensor cores, forward and
// gradient: bf16 io, head sizes 64 and 128, 128-token chunks.
//
// Chunk (g = running log decay inside it, G_ij = exp(g_i - g_j) for j <= i, A =
// SL(K K^T . G); X = S^T, the state before the chunk; D = its adjoint, transposed,
// behind the chunk):
//   T' = (I + A diag(beta))^-1       T = (I + diag(beta) A)^-1
// forward, the prediction errors e and written rows u = beta e:
//   e = T' V - [T' diag(exp(g)) K] X = U - W X
//   X <- exp(g_C) X + K^T diag(exp(g_C - g)) u
//   O = scale (diag(exp(g)) Q X + (Q K^T . G) u)
// backward, w_t = D_t k_t at every token:
//   w = T^T P^T dO + [T^T diag(exp(g_C - g)) K] D = w0 + Wd D,   P = scale (Q K^T . G)
//   D <- exp(g_C) D + Bc - K^T diag(beta exp(g)) w,   Bc = scale Q^T diag(exp(g)) dO
// so both directions are one kind of scan: a row matrix from a product with the
// state, the state from a product with the rows.  Kernels: the preparation (W, U;
// Wd, w0, Bc; parallel over chunks), the scans (sequential over a sequence's
// chunks, parallel over heads and slices of 32 d_v columns), and the outputs or
// gradients (parallel over chunks; formulas of the latter in gdr_grad.cu).
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "gdr_tc.cuh"

namespace llattn {

namespace {

using namespace gdrtc;

constexpr int kParts = 18, kBnd = 64;
// per (chunk, head)
struct Tables {
  float2 g[kC];    // running log decay
  float into[kC];  // exp(g_t) (of the gradient)
  float rel[kC];   // exp(g_t - g_0): what D takes from a chunk all carries exp(g_0), which may be tiny
  float p[kC];     // inverse scales of the rows of the fp16 tile of K
  float out[kC];   // exp(g_C - g_t)
  float row[kC];   // beta p: what makes u' and p beta w of e and w
  float4 all;      // what exp(g_C) is made of (below), exp(g_0), eps
  float iq, id;    // inverse scales of the fp16 tiles of Q and dO
  unsigned mu, mw; // bits of the largest element of the rows u' and p beta w (of the gradient)
};

struct TcParams {
  GdrSeqs seqs;
  int dk, dv, slots;
  float scale;
  const __nv_bfloat16 *q, *k, *v, *dout;
  const float *log_alpha, *beta, *state_in, *dstate_out;
  __nv_bfloat16 *o, *dq, *dkey, *dval;
  float *state_out, *dstate_in, *dlog_alpha, *dbeta;
  // workspace, per (slot, head) unless said otherwise; tiles are fp16
  unsigned char* W;      // two tiles, [token][d_k]
  float* U;              // [slice of 32][piece of 4][token][4]; the scan for the gradient leaves e there
  unsigned char* K16;    // per (slot, key head), a scale to each row
  unsigned char* S;      // X before the chunk, scaled: a tile [d_k][d_v]; for the gradient slice tiles
  unsigned char* E;      // p eps u, scaled: a tile [token][d_v]; likewise
  Tables* tab;
  unsigned *amax_s, *amax_d;  // [sequence, head]: bits of the largest value that scales X and e, D and w
  // the gradient's
  unsigned char *Q16, *dO16;  // Q16 per (slot, key head)
  unsigned char* Wd;
  float *w0, *Bc;        // as U, Bc's rows being d_k
  unsigned char* D;      // D behind the chunk, scaled: a tile [d_k][d_v]
  unsigned char* Y;      // p eps beta w, scaled: a tile [token][d_v]
  float* final_state;    // [sequence, head, dv, dk]
  float2* part;          // [16][token]: e.w and v.(beta w) over 8 columns; then [4][token] floats, parts of q.dq
  float* bnd;            // [kBnd]: pieces of <S, D> behind the chunk
  unsigned* err;
};

// ---------------------------------------------------------------- preparation
__device__ __forceinline__ float4 chunk_factors(const float2* gs, float eps) {
  const float2 g0 = gs[0], g = gs[kC - 1];
  const float d = g.x + g.y;
  return make_float4(d > -0.5f ? expm1f(d) : 0.f, d > -0.5f ? -1.f : expf(d), gdr_alpha(g0.x + g0.y), eps);
}
// exp(g_C), by which the state is multiplied chunk after chunk: what the product of the rounded
// factors so far is off by, `off` (relative), is taken out of one near 1 before that is rounded, so that
// roundings which repeat do not add up (log alpha = -1.3e-6: 3e-8 a chunk, 3e-5 after 131072 tokens).
__device__ __forceinline__ float chunk_decay(float4 all, float& off) {
  const float c = all.x - off, r = 1.f + c;
  off = (r - 1.f) - c;
  return all.y < 0.f ? r : all.y;
}
// one (chunk, head): its number (no more when it is the item count), sequence, place and length
struct Item {
  int it, seq, chunk, t0, n, len;
  size_t row0, krow0;
};
// the first item at or after `it`, `step` apart, that a chunk owns
__device__ __noinline__ void find_item(const TcParams& p, int it, int step, Item* out) {
  const int items = p.slots * p.seqs.H;
  for (; it < items; it += step) {
    const int slot = it / p.seqs.H, h = it - slot * p.seqs.H, hk = h / (p.seqs.H / p.seqs.Hk);
    int seq, chunk;
    GdrSeq sq;
    if (!gdr_find(p.seqs, slot, kC, seq, chunk, sq)) continue;
    out->seq = seq;
    out->chunk = chunk;
    out->t0 = chunk * kC;
    out->n = min(kC, sq.len - chunk * kC);
    out->len = sq.len;
    out->row0 = ((size_t)sq.row_b * p.seqs.H + h) * p.seqs.T + sq.start + chunk * kC;
    out->krow0 = ((size_t)sq.row_b * p.seqs.Hk + hk) * p.seqs.T + sq.start + chunk * kC;
    break;
  }
  out->it = it;
}
// likewise of (chunk, key head): number slot Hk + head, row0 that of its first value head
__device__ __noinline__ void find_unit(const TcParams& p, int it, int step, Item* out) {
  const int units = p.slots * p.seqs.Hk;
  for (; it < units; it += step) {
    const int slot = it / p.seqs.Hk, hk = it - slot * p.seqs.Hk, h = hk * (p.seqs.H / p.seqs.Hk);
    int seq, chunk;
    GdrSeq sq;
    if (!gdr_find(p.seqs, slot, kC, seq, chunk, sq)) continue;
    out->seq = seq;
    out->chunk = chunk;
    out->t0 = chunk * kC;
    out->n = min(kC, sq.len - chunk * kC);
    out->len = sq.len;
    out->row0 = ((size_t)sq.row_b * p.seqs.H + h) * p.seqs.T + sq.start + chunk * kC;
    out->krow0 = ((size_t)sq.row_b * p.seqs.Hk + hk) * p.seqs.T + sq.start + chunk * kC;
    break;
  }
  out->it = it;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

struct PrepSm {
  static constexpr uint32_t kX0 = 0;                               // K (forward: of every other chunk)
  static constexpr uint32_t kX1 = kTile;                           // Q (forward: K of the others)
  static constexpr uint32_t kX2 = 2 * kTile;                       // V; backward then dO
  static constexpr uint32_t kM = 3 * kTile;                        // M, float32; then operands in two parts
  static constexpr uint32_t kR = kM + kMatB;                       // A, float32; then likewise
  static constexpr uint32_t kTab = kR + 2 * kTile;
  static constexpr uint32_t kCol = kTab + 4 * kC * 4 + 32 + 64 + 16;  // forward: the columns' decay factors
  static constexpr uint32_t kBars = kCol + kColDecays * 4;
  static_assert(kBars >= kTab + 5 * kC * 4 + 32 + 4 * 64 + 16, "the backward's tables");
  static constexpr uint32_t kNext = kBars + 7 * 8;
  static constexpr uint32_t kBytes = kNext + 2 * sizeof(Item);
  static_assert(kCol % 16 == 0, "read as float4");
};
static_assert(kMatB == 2 * kTile && PrepSm::kBars % 8 == 0, "tile alignment");
static_assert(PrepSm::kBytes <= 232448, "shared memory budget of one CTA");
struct TcMaps {  // [rows, d] bf16, boxes of 64 columns and 128 rows
  CUtensorMap q, k, v, dout;
};

constexpr float kScoreDown = 1.f / 1024.f;  // of the scores Q K^T of scaled tiles, as operands
constexpr float kKeysDown = 1.f / 1024.f;  // of K K^T of the scaled rows (at most 128 x 64^2)
constexpr float kRowsDown = 1.f / 16.f;    // of P^T dO, as an operand

// Both are persistent, one CTA per SM, an item per (chunk, head).  Thread = (row,
// quarter of the columns); while warps 0 to 7 solve for M, the others prepare
// what is needed next.  The latency of an item's chain bounds them, the solve half
// of it: seven tiles fill the shared memory, so that no second item is in
// work beside it.  Measured: forward 13.5 us an item and SM (183 us for 2048 items),
// backward 29 (195 us for 1024), 2.8 TB/s of its own traffic.
constexpr int kPrepThreads = 512, kPrepBar2 = 2;

// The forward's.  Warps 8 to 15 make V's operand and, a whole item ahead, everything
// of the next chunk up to K K^T.
__global__ void __launch_bounds__(kPrepThreads, 1)
    gdr_prep_fwd_kernel(const __grid_constant__ TcMaps maps, TcParams p) {
  using Sm = PrepSm;
  extern __shared__ __align__(1024) unsigned char s[];
  let_next_launch();
  if (smem_u32(s) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceArg);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, qt = warp >> 2;
  const int i = 32 * q + lane;  // this thread's row (TMEM lane), columns 32 qt ..
  float2* gs = reinterpret_cast<float2*>(s + Sm::kTab);
  float* bs = reinterpret_cast<float*>(gs + kC);
  float* in_s = bs + kC;
  float2* tot = reinterpret_cast<float2*>(in_s + kC);
  uint32_t* red = reinterpret_cast<uint32_t*>(tot + 4);  // 2 x 8
  float* inv = reinterpret_cast<float*>(red + 16);       // inverse scales of V and of p_all
  float* cf = reinterpret_cast<float*>(s + Sm::kCol);
  uint64_t* bar = reinterpret_cast<uint64_t*>(s + Sm::kBars);  // K K^T, U, W, K loads 0 and 1, V load
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + Sm::kBars + 6 * 8);
  Item* next = reinterpret_cast<Item*>(s + Sm::kNext);
  float* Ap = reinterpret_cast<float*>(s + Sm::kR);
  float* Mp = reinterpret_cast<float*>(s + Sm::kM);
  unsigned char *M = s + Sm::kM, *X0 = s + Sm::kX0, *XV = s + Sm::kX2, *R = s + Sm::kR;
  const uint32_t sX0 = smem_u32(X0), sXV = smem_u32(XV), sR = smem_u32(R), sM = smem_u32(M);
  const int items = p.slots * p.seqs.H, G = p.seqs.H / p.seqs.Hk;
  if (tid == 0) {
    for (int b = 0; b < 6; ++b) mbar_init(bar + b, 1);
    fence_mbar_init();
    find_item(p, blockIdx.x, gridDim.x, next);
    find_item(p, next->it + gridDim.x, gridDim.x, next + 1);
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + 32 * qt;

  const int t = tid - 256;  // of the threads of warps 8 to 15
  float beta_n = 0.f, p_n = 1.f, all_n = 1.f;  // beta, scaled, and p of the next item's token t / 2, p_all
  auto load_k = [&](const Item& x, int b) { load_tile(X0 + b * kTile, &maps.k, (int)x.krow0, bar + 3 + b); };
  // decays, K's operand and K K^T of item x, number j of this CTA (warps 8 to 15)
  auto stage_keys = [&](const Item& x, int j) {
    const int b = j & 1, slot = x.it / p.seqs.H, h = x.it - slot * p.seqs.H;
    const float la = t < x.n ? gdr_log(p.log_alpha[x.row0 + t]) : 0.f;
    const float bt = t / 2 < x.n ? p.beta[x.row0 + t / 2] : 0.f;
    chunk_decays(la, gs, tot, t, kPrepBar2, 256);
    column_decays(cf, gs, t);
    wait_bar(bar + 3 + b, (j >> 1) & 1, p.err);
    const Keys key = keys_to_f16<256>(X0 + b * kTile, x.n, red, t, kPrepBar2);
    p_n = key.p;
    all_n = key.p_all;
    // A is K K^T of the scaled rows, beta takes the scales
    beta_n = bt * p_n * p_n / kKeysDown;
    Tables& tb = p.tab[x.it];
    uint32_t* bounds = reinterpret_cast<uint32_t*>(tot);  // (the decays' sums have been read)
    const uint32_t most = __reduce_max_sync(0xffffffffu, rows_bound(bt, p_n, key.l1));
    if (lane == 0) bounds[warp - 8] = most;
    if ((t & 1) == 0) {
      tb.p[t / 2] = p_n;
      tb.row[t / 2] = bt * p_n;
    }
    if (t < kC) {
      const float2 g = gs[t];
      tb.g[t] = g;
      tb.out[t] = exp_diff(gs[kC - 1], g);
    }
    tc_fence_before();
    named_bar_sync(kPrepBar2, 256);
    if (t == 32) tb.all = chunk_factors(gs, rows_scale(max_of<8>(bounds)));
    if (t == 0) {
      tc_fence_after();
      mma_tile<kAlong, kAlong>(tmem, sX0 + b * kTile, sX0 + b * kTile, false);
      umma_commit(bar);
      if (h % G == 0) {
        bulk_store(p.K16 + ((size_t)slot * p.seqs.Hk + h / G) * kTile, X0 + b * kTile, kTile);
        bulk_commit();
      }
    }
    __syncwarp();
  };

  Item me = next[0];
  if (me.it < items) {
    if (t == 0) {
      load_k(me, 0);
      load_tile(XV, &maps.v, (int)me.row0, bar + 5);
      if (next[1].it < items) load_k(next[1], 1);
    }
    __syncwarp();
    if (warp >= 8) stage_keys(me, 0);
  }
  for (int j = 0; me.it < items; ++j) {
    const int it = me.it, b = j & 1;
    const int slot = it / p.seqs.H, h = it - slot * p.seqs.H;
    const size_t sh = (size_t)me.seq * p.seqs.H + h;
    wait_bar(bar, j & 1, p.err);
    __syncwarp();
    tc_fence_after();
    if (tid == 0) bulk_wait_read1();  // U of the item before has left
    __syncthreads();
    const Item nx = next[b ^ 1];
    const float2 gi = gs[i];
    const float pi = p.tab[it].p[i];
    if (t >= 0 && (t & 1) == 0) bs[t / 2] = beta_n;
    if (t >= 0 && t < kC) in_s[t] = exp_diff(gs[t], make_float2(0.f, 0.f));
    // A_ij = (k_i . k_j) G_ij, j < i
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      const int j0 = 32 * qt + 16 * c;
      if (j0 > 32 * q + 31) break;  // (warp-uniform) above the diagonal
      float x[16];
      decayed16(x, tl + 16 * c, cf, gs, gi, i, q, j0, i, kKeysDown);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        mat4(Ap, i, (j0 >> 2) + v) = make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
    }
    if (tid == 0) bulk_wait_read0();  // and W
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp < 8) {
      tri_solve(Ap, Mp, bs, tid);
    } else {
      wait_bar(bar + 5, j & 1, p.err);
      uint32_t vbits;
      const float iv = values_to_f16<256>(XV, me.n, p_n * pow2_inverse(all_n), red + 8, t, kPrepBar2, &vbits);
      if (lane == 0) atomicMax(p.amax_s + sh, vbits);
      if (t == 0) {
        inv[0] = iv;
        inv[1] = pow2_inverse(all_n);
      }
      if (p.state_in && me.chunk == 0) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, state_max(p.state_in + sh * p.dv * p.dk, p.dv * p.dk, t, 256));
        if (lane == 0) atomicMax(p.amax_s + sh, m);
      }
      if (nx.it < items) {
        stage_keys(nx, j + 1);
        if (t == 255) {  // the item after the next, V of the next on its way into L2
          find_item(p, nx.it + gridDim.x, gridDim.x, next + b);
          bulk_prefetch_l2(p.v + nx.row0 * p.dv, (uint32_t)(nx.n * p.dv * 2));
        }
      }
    }
    __syncthreads();
    // ---- U = T' V -> 256, W = T' diag(exp(g)) K -> 384 (of v' and k', a row's p in the end)
    const float iv = inv[0] * (pi * inv[1]);
    float m[32];
    load_m(m, Mp, i, qt);
    __syncthreads();
    put_inverse2(R, M, m, i, qt, bs, in_s);
    fence_proxy_async_shared();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      mma_tile<kAlong, kDown>(tmem + 256, sR + kTile, sXV, false);
      mma_tile<kAlong, kDown>(tmem + 256, sR, sXV, true);
      umma_commit(bar + 1);
      mma_tile<kAlong, kDown>(tmem + 384, sM + kTile, sX0 + b * kTile, false);
      mma_tile<kAlong, kDown>(tmem + 384, sM, sX0 + b * kTile, true);
      umma_commit(bar + 2);
    }
    __syncwarp();
    wait_bar(bar + 1, j & 1, p.err);
    __syncwarp();
    tc_fence_after();
    if (t == 0 && nx.it < items) load_tile(XV, &maps.v, (int)nx.row0, bar + 5);
    __syncwarp();
    // U and W leave by way of the operands' places
    write_rows(reinterpret_cast<float*>(R), tl + 256, i, qt, iv / kInvUp);
    fence_proxy_async_shared();
    __syncthreads();
    if (tid == 0) {
      bulk_store(p.U + (size_t)it * kC * kC, R, kMatB);
      bulk_commit();
    }
    __syncwarp();
    wait_bar(bar + 2, j & 1, p.err);
    __syncwarp();
    tc_fence_after();
    if (t == 0 && nx.it < items && next[b].it < items) {
      bulk_wait_read0();  // this item's K16 (and the next one's)
      load_k(next[b], b);
    }
    __syncwarp();
    write_tiles<true>(M, M + kTile, tl + 384, i, qt, pi / kInvUp, kLoScale);
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      bulk_store(p.W + (size_t)it * 2 * kTile, M, 2 * kTile);
      bulk_commit();
    }
    __syncwarp();
    me = nx;
  }
  if (tid == 0 || t == 0) bulk_wait0();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The backward's.  Products are issued by thread 0, which they hold for as long as they
// run (about 100 cycles each); with a warp of its own for that, 544 threads leave 96
// registers each, and an item took 31 us.
__global__ void __launch_bounds__(kPrepThreads, 1)
    gdr_prep_bwd_kernel(const __grid_constant__ TcMaps maps, TcParams p) {
  using Sm = PrepSm;
  extern __shared__ __align__(1024) unsigned char s[];
  let_next_launch();
  if (smem_u32(s) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceArg);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, qt = warp >> 2;
  const int i = 32 * q + lane;  // this thread's row (TMEM lane), columns 32 qt ..
  float2* gs = reinterpret_cast<float2*>(s + Sm::kTab);
  float* bs = reinterpret_cast<float*>(gs + kC);
  float* in_s = bs + kC;
  float* out_s = in_s + kC;
  float2* tot = reinterpret_cast<float2*>(out_s + kC);
  uint32_t* red = reinterpret_cast<uint32_t*>(tot + 4);  // 3 x 16
  float* inv = reinterpret_cast<float*>(red + 48);       // inverse scales of V, Q and of p_all
  uint32_t* bounds = red + 52;                           // 16
  float* cf = reinterpret_cast<float*>(s + Sm::kM);  // the columns' decay factors, where M comes to stand
  uint64_t* bar = reinterpret_cast<uint64_t*>(s + Sm::kBars);
  // bar: products, K, U, Q, V and dO, Q K^T
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + Sm::kBars + 6 * 8);
  Item* next = reinterpret_cast<Item*>(s + Sm::kNext);
  float* Ap = reinterpret_cast<float*>(s + Sm::kR);
  float* Mp = reinterpret_cast<float*>(s + Sm::kM);
  unsigned char* M = s + Sm::kM;
  unsigned char *X0 = s + Sm::kX0, *X1 = s + Sm::kX1, *XV = s + Sm::kX2, *R = s + Sm::kR;
  const uint32_t sX0 = smem_u32(X0), sX1 = smem_u32(X1), sXV = smem_u32(XV), sR = smem_u32(R),
                 sM = smem_u32(M);
  if (tid == 0) {
    for (int b = 0; b < 6; ++b) mbar_init(bar + b, 1);
    fence_mbar_init();
    find_item(p, blockIdx.x, gridDim.x, next);
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + 32 * qt;
  uint32_t nmma = 0, items_done = 0;
  auto wait_mma = [&]() {
    wait_bar(bar, nmma & 1, p.err);
    ++nmma;
    __syncwarp();
    tc_fence_after();
  };
  // operands in shared memory are ready: thread 0 issues the products
  auto issue = [&](auto products) {
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      products();
      umma_commit(bar);
    }
    __syncwarp();
  };
  auto raise_max = [&](unsigned* at, uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) atomicMax(at, m);
  };

  const int items = p.slots * p.seqs.H, G = p.seqs.H / p.seqs.Hk;
  float la = 0.f, bt = 0.f;  // this thread's token's, of the item that is loaded
  auto load_keys = [&](const Item& x) {
    if (tid == 0) {
      load_tile(X0, &maps.k, (int)x.krow0, bar + 1);
      load_tile(X1, &maps.q, (int)x.krow0, bar + 3);
    }
    __syncwarp();
    la = tid < x.n ? p.log_alpha[x.row0 + tid] : 0.f;  // (not used before the next item)
    bt = tid < x.n ? p.beta[x.row0 + tid] : 0.f;
  };
  uint32_t nv = 0, nkq = 0;  // loads of V and dO, and of K, waited for
  auto load_values = [&](const CUtensorMap* map, size_t row, int by) {
    if (tid == by) load_tile(XV, map, (int)row, bar + 4);
    __syncwarp();
  };
  Item me = *next;
  if (me.it < items) {
    load_keys(me);
    load_values(&maps.v, me.row0, 0);
  }
  while (me.it < items) {
    const int it = me.it, n = me.n;
    const int slot = it / p.seqs.H, h = it - slot * p.seqs.H, hk = h / G;
    const size_t row0 = me.row0, sh = (size_t)me.seq * p.seqs.H + h;
    unsigned* am_s = p.amax_s + sh;
    Tables& tb = p.tab[it];
    unsigned char* Wg = p.W + (size_t)it * 2 * kTile;
    unsigned char* Wdg = p.Wd + (size_t)it * 2 * kTile;
    const bool t_end = me.t0 + n == me.len;
    if (tid < kC) bs[tid] = bt;
    chunk_decays(gdr_log(la), gs, tot, tid, 0, kPrepThreads);
    column_decays(cf, gs, tid);
    const float2 gi = gs[i];
    if (qt == 0) {
      const float in = exp_diff(gi, make_float2(0.f, 0.f)), out = exp_diff(gs[kC - 1], gi);
      in_s[i] = in;
      out_s[i] = out;
      tb.g[i] = gi;
      tb.into[i] = gdr_alpha(gi.x + gi.y);
      tb.out[i] = out;
      tb.rel[i] = exp_diff(gi, gs[0]);
    }
    if (p.state_in && me.chunk == 0) raise_max(am_s, state_max(p.state_in + sh * p.dv * p.dk, p.dv * p.dk, tid, kPrepThreads));
    wait_bar(bar + 1, nkq & 1, p.err);
    const Keys key = keys_to_f16<kPrepThreads>(X0, n, red, tid, 0);
    if (tid == 0) inv[2] = pow2_inverse(key.p_all);
    // ---- K K^T -> 0
    issue([&]() {
      mma_tile<kAlong, kAlong>(tmem, sX0, sX0, false);
      bulk_wait_read0();  // (what the item before staged has left)
      if (h % G == 0) {
        bulk_store(p.K16 + ((size_t)slot * p.seqs.Hk + hk) * kTile, X0, kTile);
        bulk_commit();
      }
    });
    {  // A is K K^T of the scaled rows, beta takes the scales
      const float bk = bs[tid / 4], pk = key.p;
      const uint32_t most = __reduce_max_sync(0xffffffffu, rows_bound(bk, pk, key.l1));
      if (lane == 0) bounds[warp] = most;
      if ((tid & 3) == 0) {
        bs[tid / 4] = bk * pk * pk / kKeysDown;
        tb.p[tid / 4] = pk;
        tb.row[tid / 4] = bk * pk;
      }
    }
    wait_mma();
    // A_ij = (k_i . k_j) G_ij, j < i
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      const int j0 = 32 * qt + 16 * c;
      if (j0 > 32 * q + 31) break;  // (warp-uniform) above the diagonal
      float x[16];
      decayed16(x, tl + 16 * c, cf, gs, gi, i, q, j0, i, kKeysDown);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        mat4(Ap, i, (j0 >> 2) + v) = make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
    }
    __syncthreads();
    const float pi = tb.p[i];
    if (warp < 8) {
      tri_solve(Ap, Mp, bs, tid);
    } else {
      const int t = tid - 256;
      uint32_t vbits;
      const float pv = tb.p[t / 2];
      if (t == 0) {
        tb.all = chunk_factors(gs, rows_scale(max_of<16>(bounds)));
        tb.mu = tb.mw = 0u;
      }
      wait_bar(bar + 4, nv & 1, p.err);
      const float iv = values_to_f16<256>(XV, n, pv * inv[2], red + 16, t, kPrepBar2, &vbits);
      if (lane == 0) atomicMax(am_s, vbits);
      wait_bar(bar + 3, nkq & 1, p.err);
      const float iq = tile_to_f16<256>(X1, n, red + 32, t, kPrepBar2);
      tc_fence_before();
      named_bar_sync(kPrepBar2, 256);
      if (t == 0) {  // Q K^T -> 128, while the tensor cores are free
        tc_fence_after();
        mma_tile<kAlong, kAlong>(tmem + 128, sX1, sX0, false);
        umma_commit(bar + 5);
        inv[0] = iv;
        inv[1] = iq;
        tb.iq = iq;
      }
      if (warp == 15) {  // the next item: where it is, and its rows on their way into L2
        if (lane == 0) find_item(p, it + gridDim.x, gridDim.x, next);
        __syncwarp();
        if (next->it < items) {
          const char* kp = reinterpret_cast<const char*>(p.k + next->krow0 * p.dk);
          const char* qp = reinterpret_cast<const char*>(p.q + next->krow0 * p.dk);
          const char* vp = reinterpret_cast<const char*>(p.v + next->row0 * p.dv);
          const char* dp = reinterpret_cast<const char*>(p.dout + next->row0 * p.dv);
          for (int x = lane * 128; x < next->n * p.dk * 2; x += 32 * 128) {
            prefetch_l2(kp + x);
            prefetch_l2(qp + x);
          }
          for (int x = lane * 128; x < next->n * p.dv * 2; x += 32 * 128) {
            prefetch_l2(vp + x);
            prefetch_l2(dp + x);
          }
          if (lane * 32 < next->n) {
            prefetch_l2(p.log_alpha + next->row0 + lane * 32);
            prefetch_l2(p.beta + next->row0 + lane * 32);
          }
        }
      }
    }
    __syncthreads();
    me = *next;
    ++nv;
    ++nkq;
    const float iv = inv[0] * (pi * inv[2]), iq = inv[1], bi = bs[i];
    // ---- U = T' V -> 256, W = T' diag(exp(g)) K -> 384 (of v' and k', a row's p in the end)
    float m[32];
    load_m(m, Mp, i, qt);
    __syncthreads();
    put_inverse2(R, M, m, i, qt, bs, in_s);
    issue([&]() {
      mma_tile<kAlong, kDown>(tmem + 256, sR + kTile, sXV, false);
      mma_tile<kAlong, kDown>(tmem + 256, sR, sXV, true);
      umma_commit(bar + 2);
      mma_tile<kAlong, kDown>(tmem + 384, sM + kTile, sX0, false);
      mma_tile<kAlong, kDown>(tmem + 384, sM, sX0, true);
      if (h % G == 0) {
        bulk_store(p.Q16 + ((size_t)slot * p.seqs.Hk + hk) * kTile, X1, kTile);
        bulk_commit();
      }
    });
    wait_bar(bar + 2, items_done++ & 1, p.err);
    __syncwarp();
    tc_fence_after();
    {
      load_values(&maps.dout, row0, 256);  // (V has been read; thread 0 may still be issuing products)
      write_rows(p.U + (size_t)it * kC * kC, tl + 256, i, qt, iv / kInvUp);
      const float rel = exp_diff(gi, gs[0]), in0 = in_s[0];
      // ---- Wd = T^T diag(exp(g_C - g)) K -> 0, Bc = Q^T diag(exp(g)) dO -> 256 (exp(g_0) and its scales below)
      put_inverse(R, R + kTile, m, i, qt, out_s[i], bi);
      wait_mma();
      wait_bar(bar + 4, nv & 1, p.err);
      ++nv;
      const float id = tile_to_f16<kPrepThreads>(XV, n, red, tid, 0);
      __syncthreads();
      column_decays(bs, gs, tid);  // (the tables' values have been read)
#pragma unroll 1
      for (int c8 = 0; c8 < 4; ++c8) {
        const uint32_t at = swz16(i, 4 * qt + c8);
        const uint4 v = *reinterpret_cast<const uint4*>(XV + at);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_f16x2(w[e]);
          x[2 * e] = rel * f.x;
          x[2 * e + 1] = rel * f.y;
        }
        put_parts(M, M + kTile, at, x, 1.f);
      }
      issue([&]() {
        mma_tile<kDown, kDown>(tmem, sR + kTile, sX0, false);
        mma_tile<kDown, kDown>(tmem, sR, sX0, true);
        mma_tile<kDown, kDown>(tmem + 256, sX1, sM + kTile, false);
        mma_tile<kDown, kDown>(tmem + 256, sX1, sM, true);
        bulk_store(p.dO16 + (size_t)it * kTile, XV, kTile);
        bulk_commit();
        tb.id = id;
      });
      write_tiles<true>(Wg, Wg + kTile, tl + 384, i, qt, pi / kInvUp, kLoScale);
      if (tid == 0) bulk_wait_read0();  // K16, Q16, dO16
      wait_mma();
      // ---- P^T dO -> 384
      wait_bar(bar + 5, (nkq - 1) & 1, p.err);
      __syncwarp();
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        float x[16];
        const int j0 = 32 * qt + 16 * c;
        decayed16(x, tl + 128 + 16 * c, bs, gs, gi, i, q, j0, i + 1, kScoreDown);
        put_parts(R, R + kTile, swz16(i, j0 >> 3), x, 1.f);
        put_parts(R, R + kTile, swz16(i, (j0 >> 3) + 1), x + 8, 1.f);
      }
      issue([&]() {
        mma_tile<kDown, kDown>(tmem + 384, sR + kTile, sXV, false);
        mma_tile<kDown, kDown>(tmem + 384, sR, sXV, true);
      });
      const bool last = p.dstate_out && t_end;
      if (me.it < items) {  // K and Q have been read
        load_keys(me);
      }
      write_tiles<true>(Wdg, Wdg + kTile, tl, i, qt, pi / kInvUp, kLoScale);
      wait_mma();
      // ---- w0 = T^T (P^T dO) -> 0
      put_inverse(R, R + kTile, m, i, qt, 1.f, bi);
      write_tiles<false>(M, M + kTile, tl + 384, i, qt, kRowsDown, 1.f);
      issue([&]() {
        mma_tile<kDown, kDown>(tmem, sR + kTile, sM, false);
        mma_tile<kDown, kDown>(tmem, sR, sM + kTile, true);
        mma_tile<kDown, kDown>(tmem, sR, sM, true);
      });
      if (me.it < items) {
        load_values(&maps.v, me.row0, 0);
      }
      uint32_t mx = write_rows(p.Bc + (size_t)it * kC * kC, tl + 256, i, qt, p.scale * iq * id * in0);
      if (last) mx = max(mx, state_max(p.dstate_out + sh * p.dv * p.dk, p.dv * p.dk, tid, kPrepThreads));
      wait_mma();
      mx = max(mx, write_rows(p.w0 + (size_t)it * kC * kC, tl, i, qt,
                              p.scale * iq * pi * id / (kScoreDown * kRowsDown * kInvUp)));
      raise_max(p.amax_d + sh, mx);
    }
    tc_fence_before();  // (for the next item's products, behind its barriers)
  }
  if (tid == 0) bulk_wait0();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- scan
// Slice tiles: for each slice of 32 d_v columns a [128 rows][high 32 | low 32] block
// of 16 KB, as a scan's operands stand in shared memory, from where the copy
// engine takes them to the workspace.
enum ScanMode : int { kFwd, kFwdKeep, kRev };  // the forward; the forward for the gradient; backwards
template <int MODE> struct ScanSm {
  static constexpr bool kLean = MODE != kFwd;                 // one W and one K, and room for staged rows
  static constexpr uint32_t kW = 0;                           // W (Wd), two parts (of two chunks)
  static constexpr uint32_t kK = kW + (kLean ? 2 : 4) * kTile;  // K (of two chunks)
  static constexpr uint32_t kX = kK + (kLean ? 1 : 2) * kTile;  // X (D)
  static constexpr uint32_t kE = kX + kHalf;                  // the rows as an operand
  static constexpr uint32_t kRows = kE + kHalf;               // U (w0) of two chunks: [piece of 4][token][4]
  static constexpr uint32_t kErr = kRows + 2 * kHalf;         // e, on its way out or in
  static constexpr uint32_t kU = kErr + kHalf;                // u on its way out
  static constexpr uint32_t kBc = kErr + kHalf;               // backwards: Bc
  static constexpr uint32_t kSt = kBc + kHalf;                // S of the chunk behind
  static constexpr uint32_t kBars = MODE == kFwd ? kRows : MODE == kFwdKeep ? kU + kHalf : kSt + kHalf;
  static constexpr uint32_t kBytes = kBars + 96;
  static_assert(kBytes <= 232448, "shared memory budget of one CTA");
};
enum ScanBar : int { SB_W0 = 0, SB_W1, SB_K0, SB_K1, SB_R0, SB_R1, SB_ERR, SB_BC, SB_ST, SB_MMA, kScanBars };

// One CTA per (32 d_v columns, head, sequence); thread = (TMEM lane, 8 of the
// columns), the lane a token of the chunk or a d_k row of X in turn.  X stays
// in float32 registers; per chunk two rounds of products, W [Xh | Xl] and
// K^T [uh | ul] (the parts side by side as N = 64: the 128-row operand, which
// shared memory feeds at 128 bytes a cycle, is read once for both).  The chain of
// a chunk is what bounds it: a warp of its own issues products and copies, and
// what does not belong to the chain is done in the products' time.  With most of
// the SM's memory taken as shared memory, little is left for loads in flight
// through L1 (72 KB of them a chunk took 4 thousand cycles to issue): the modes
// with many rows have them copied into shared memory instead.  Measured per chunk:
// forward 1.70 us (218 us for 128 chunks of 16 heads, 64 CTAs); with 128 CTAs,
// for the gradient 2.4 us forwards and 3.2 backwards, whose rows and tiles, 350 and 510 KB
// a chunk and head, go at 4.8 and 5.2 TB/s.
constexpr int kScanThreads = 512 + 32;
constexpr int kScanBarX = 1, kScanBarE = 2, kScanBarU = 3;  // named barriers: an operand, the staged rows are ready
template <int MODE>
__global__ void __launch_bounds__(kScanThreads, 1) gdr_scan_kernel(TcParams p, int slices) {
  constexpr bool REV = MODE == kRev, LEAN = MODE != kFwd;
  using Sm = ScanSm<MODE>;
  extern __shared__ __align__(1024) unsigned char s[];
  wait_for_previous();
  let_next_launch();
  if (smem_u32(s) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceArg);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, qt = (warp >> 2) & 3, i = 32 * q + lane;
  const int sl = blockIdx.x % slices, h = (blockIdx.x / slices) % p.seqs.H, seq = gdr_pick(p.seqs, blockIdx.x / slices / p.seqs.H);
  GdrSeq sq;
  if (!gdr_seq(p.seqs, seq, sq)) {
    if (tid == 0) raise_error(p.err, kErrDeviceArg);
    return;
  }
  const int hk = h / (p.seqs.H / p.seqs.Hk);
  const int col0 = kSlice * sl + 8 * qt;  // this thread's first d_v column
  const bool cols_in = warp < 16 && col0 < p.dv;
  const int Nc = (sq.len + kC - 1) / kC;
  const int base = gdr_slot_base(p.seqs, seq, sq.start, kC);
  const size_t row0 = ((size_t)sq.row_b * p.seqs.H + h) * p.seqs.T + sq.start;
  const size_t sh = (size_t)seq * p.seqs.H + h;
  auto item = [&](int c) { return (size_t)(base + c) * p.seqs.H + h; };
  auto at_step = [&](int x) { return REV ? Nc - 1 - x : x; };  // the chunk of step x
  auto slice_of = [&](int x) { return (item(at_step(x)) * 4 + sl) * kHalf; };  // in bytes: slice tiles, rows

  const float* from = REV ? p.dstate_out : p.state_in;
  float X[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) X[j] = from && i < p.dk && cols_in ? from[(sh * p.dv + col0 + j) * p.dk + i] : 0.f;

  uint64_t* bars = reinterpret_cast<uint64_t*>(s + Sm::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + Sm::kBars + kScanBars * 8);
  auto copy_in = [&](int bar, uint32_t at, const void* src, uint32_t bytes) {
    mbar_arrive_expect_tx(bars + bar, bytes);
    bulk_load(s + at, src, bytes, bars + bar);
  };
  auto load_w = [&](int x) {
    const int b = LEAN ? 0 : x & 1;
    copy_in(SB_W0 + b, Sm::kW + b * 2 * kTile, (REV ? p.Wd : p.W) + item(at_step(x)) * 2 * kTile, 2 * kTile);
  };
  auto load_k = [&](int x) {
    const int b = LEAN ? 0 : x & 1;
    copy_in(SB_K0 + b, Sm::kK + b * kTile, p.K16 + ((size_t)(base + at_step(x)) * p.seqs.Hk + hk) * kTile, kTile);
  };
  auto bytes_of = [&](float* x) { return reinterpret_cast<unsigned char*>(x); };
  auto load_rows = [&](int x) {
    copy_in(SB_R0 + (x & 1), Sm::kRows + (x & 1) * kHalf, bytes_of(REV ? p.w0 : p.U) + slice_of(x), kHalf);
  };
  auto load_err = [&](int x) { copy_in(SB_ERR, Sm::kErr, bytes_of(p.U) + slice_of(x), kHalf); };
  auto load_bc = [&](int x) { copy_in(SB_BC, Sm::kBc, bytes_of(p.Bc) + slice_of(x), kHalf); };
  auto load_st = [&](int x) { copy_in(SB_ST, Sm::kSt, p.S + slice_of(x), kHalf); };
  if (tid == 0) {
    for (int b = 0; b < kScanBars; ++b) mbar_init(bars + b, 1);
    fence_mbar_init();
    for (int x = 0; x < 2 && x < Nc; ++x) {
      if (!LEAN || x == 0) {
        load_w(x);
        load_k(x);
      }
      if (LEAN) load_rows(x);
    }
    if (REV && Nc) {
      load_err(0);
      load_bc(0);
      if (Nc > 1) load_st(0);
    }
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const float2 sg =
      Nc ? operand_scale(__uint_as_float((REV ? p.amax_d : p.amax_s)[sh])) : make_float2(1.f, 1.f);
  const float isf = REV && Nc ? operand_scale(__uint_as_float(p.amax_s[sh])).y : 1.f;
  auto write_bnd = [&](int c, float d) {  // a piece of <S, D> behind chunk c
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0 && warp < 16) p.bnd[item(c) * kBnd + sl * 16 + warp] = d;
  };
  if (REV && Nc) {  // <S_T, its gradient>: what the last chunk's log decays add
    float d = 0.f;
    if (p.dstate_out && i < p.dk && cols_in)
#pragma unroll
      for (int j = 0; j < 8; ++j) d = fmaf(X[j], p.final_state[(sh * p.dv + col0 + j) * p.dk + i], d);
    write_bnd(Nc - 1, d);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) X[j] *= sg.x;

  const uint32_t tmem = *tmem_slot;
  const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + 8 * qt;
  const uint32_t sX = smem_u32(s + Sm::kX), sE = smem_u32(s + Sm::kE);
  constexpr uint32_t idW = idesc_f16(64, false, true), idK = idesc_f16(64, true, true);
  uint32_t nmma = 0;
  auto wait_mma = [&]() {
    wait_bar(bars + SB_MMA, nmma & 1, p.err);
    ++nmma;
    __syncwarp();
    tc_fence_after();
  };
  auto ready = [&](int bar) {  // this thread's part is in shared memory
    fence_proxy_async_shared();
    tc_fence_before();
    named_bar_arrive(bar, kScanThreads);
  };

  if (warp == 16) {  // products and copies
    for (int x = 0; x < Nc; ++x) {
      const int b = LEAN ? 0 : x & 1;
      const uint32_t par = (LEAN ? x : x >> 1) & 1;
      named_bar_sync(kScanBarX, kScanThreads);
      if (lane == 0) {
        if (MODE == kFwdKeep) bulk_wait_read0();  // the rows staged in the step before have left
        wait_bar(bars + SB_W0 + b, par, p.err);
        tc_fence_after();
        const uint32_t w = smem_u32(s + Sm::kW + b * 2 * kTile);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16(tmem + 64 * part, desc_of<kPlain>(w + part * kTile) + step_of<kPlain>(kk), desc_mn(sX, kk), idW, kk > 0);
        umma_commit(bars + SB_MMA);
        if (LEAN) {
          if (!REV) {
            bulk_store(p.S + slice_of(x), s + Sm::kX, kHalf);
            bulk_commit();
          }
          // rows of the step before have been read
          if (x > 0 && x + 1 < Nc) load_rows(x + 1);
          if (REV && x > 0) {
            load_err(x);
            load_bc(x);
          }
        }
      }
      __syncwarp();
      wait_mma();
      if (lane == 0) {
        if (LEAN ? x + 1 < Nc : x + 2 < Nc) load_w(LEAN ? x + 1 : x + 2);
      }
      __syncwarp();
      named_bar_sync(kScanBarE, kScanThreads);
      if (lane == 0) {
        if (REV && x > 0 && x + 1 < Nc) load_st(x);  // (the one behind has been read)
        wait_bar(bars + SB_K0 + b, par, p.err);
        if (MODE == kFwdKeep) bulk_wait_read0();  // X has left
        tc_fence_after();
        const uint32_t k = smem_u32(s + Sm::kK + b * kTile);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) umma_bf16(tmem + 128, desc_mn(k, kk), desc_mn(sE, kk), idK, kk > 0);
        umma_commit(bars + SB_MMA);
      }
      __syncwarp();
      if (MODE == kFwdKeep) {
        named_bar_sync(kScanBarU, kScanThreads);
        if (lane == 0) {
          bulk_store(p.E + slice_of(x), s + Sm::kU, kHalf);
          bulk_store(bytes_of(p.U) + slice_of(x), s + Sm::kErr, kHalf);  // e in U's place
          bulk_commit();
        }
        __syncwarp();
      }
      wait_mma();
      if (lane == 0) {
        if (LEAN ? x + 1 < Nc : x + 2 < Nc) load_k(LEAN ? x + 1 : x + 2);
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait0();
    __syncthreads();
    return;
  }

  // 8 columns of row i, times f, as high and low parts of a [row][32 | 32] tile
  const uint32_t at_hi = swz16(i, qt), at_lo = swz16(i, 4 + qt);
  auto put = [&](uint32_t tile, const float* x, float f, float lo) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = f * x[e];
    put_parts(s + tile, s + tile + (at_lo - at_hi), at_hi, y, lo);
  };
  // 8 columns of row i, times f, into a plain tile of the workspace
  auto keep = [&](unsigned char* tile, const float* x, float f) {
    *reinterpret_cast<uint4*>(tile + plain16(i, col0 >> 3)) =
        make_uint4(pack_f16x2(f * x[0], f * x[1]), pack_f16x2(f * x[2], f * x[3]), pack_f16x2(f * x[4], f * x[5]),
                   pack_f16x2(f * x[6], f * x[7]));
  };
  const uint32_t piece = (uint32_t)(2 * qt * kC + i) * 16;  // of a slice's rows, the next one 16 kC on
  auto rows8 = [&](const unsigned char* rows, float* x, float f) {
    const float4 a = *reinterpret_cast<const float4*>(rows + piece);
    const float4 b = *reinterpret_cast<const float4*>(rows + piece + 16 * kC);
    x[0] = f * a.x; x[1] = f * a.y; x[2] = f * a.z; x[3] = f * a.w;
    x[4] = f * b.x; x[5] = f * b.y; x[6] = f * b.z; x[7] = f * b.w;
  };

  // what this thread loads of a chunk itself, one step ahead
  float4 un[2];
  uint4 vn = make_uint4(0u, 0u, 0u, 0u);
  float fac_n = 0.f, row_n = 0.f, beta_n = 0.f, gam_n = 0.f, in0_n = 0.f, off = 0.f;
  auto fetch = [&](int x) {
    const int c = at_step(x), t = c * kC + i;
    if (!LEAN) {
      const unsigned char* ug = bytes_of(p.U) + slice_of(x) + piece;
      un[0] = *reinterpret_cast<const float4*>(ug);
      un[1] = *reinterpret_cast<const float4*>(ug + 16 * kC);
    }
    const Tables& tb = p.tab[item(c)];
    const float4 all = tb.all;
    const float row = tb.row[i];
    gam_n = chunk_decay(all, off);
    if (REV) in0_n = all.z;
    row_n = row * all.w;
    fac_n = row * (REV ? tb.rel[i] : tb.out[i]);
    if (REV) beta_n = t < sq.len ? p.beta[row0 + t] : 0.f;
    if (REV) vn = t < sq.len && cols_in ? *reinterpret_cast<const uint4*>(p.v + (row0 + t) * p.dv + col0)
                                        : make_uint4(0u, 0u, 0u, 0u);
  };
  if (Nc) fetch(0);
  for (int x = 0; x < Nc; ++x) {
    const int c = at_step(x);
    const size_t it = item(c);
    // ---- W X (Wd D)
    put(Sm::kX, X, 1.f, kLoScale);
    ready(kScanBarX);
    // (while the products run)
    if (MODE != kFwdKeep) keep((REV ? p.D : p.S) + it * kTile, X, 1.f);
    if (REV && x > 0) {  // <S, D> between this chunk and the one behind it: X here, that one's first state
      wait_bar(bars + SB_ST, (x - 1) & 1, p.err);
      const uint4 hv = *reinterpret_cast<const uint4*>(s + Sm::kSt + at_hi);
      const uint4 lv = *reinterpret_cast<const uint4*>(s + Sm::kSt + at_lo);
      const uint32_t hw[4] = {hv.x, hv.y, hv.z, hv.w}, lw[4] = {lv.x, lv.y, lv.z, lv.w};
      float d = 0.f;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float2 a = unpack_f16x2(hw[v]), l = unpack_f16x2(lw[v]);
        d = fmaf(X[2 * v], fmaf(kLoInv, l.x, a.x), fmaf(X[2 * v + 1], fmaf(kLoInv, l.y, a.y), d));
      }
      write_bnd(c, d * sg.y * isf);
    }
    float u[8];
    if (!LEAN) {
      u[0] = sg.x * un[0].x; u[1] = sg.x * un[0].y; u[2] = sg.x * un[0].z; u[3] = sg.x * un[0].w;
      u[4] = sg.x * un[1].x; u[5] = sg.x * un[1].y; u[6] = sg.x * un[1].z; u[7] = sg.x * un[1].w;
    } else {
      wait_bar(bars + SB_R0 + (x & 1), (x >> 1) & 1, p.err);
      rows8(s + Sm::kRows + (x & 1) * kHalf, u, sg.x);
    }
    const uint4 vr = vn;
    const float fac = fac_n, row = row_n, bt = beta_n, gam = gam_n, in0 = in0_n;
    if (x + 1 < Nc) fetch(x + 1);
    wait_mma();
    {
      float hh[8], hl[8], lh[8];
      tmem_ld8(tl, hh);
      tmem_ld8(tl + 32, hl);
      tmem_ld8(tl + 64, lh);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = fmaf(kLoInv, hl[j] + lh[j], hh[j]);
        u[j] = REV ? u[j] + y : u[j] - y;
      }
    }
    // ---- K^T (beta exp(g_C - g) e), K^T (beta exp(g - g_0) w)
    put(Sm::kE, u, fac, kLoScale);
    ready(kScanBarE);
    if (MODE == kFwdKeep) {
      put(Sm::kU, u, row, 1.f);
      float4* eg = reinterpret_cast<float4*>(s + Sm::kErr + piece);
      eg[0] = make_float4(sg.y * u[0], sg.y * u[1], sg.y * u[2], sg.y * u[3]);
      eg[kC] = make_float4(sg.y * u[4], sg.y * u[5], sg.y * u[6], sg.y * u[7]);
      ready(kScanBarU);
    } else {
      keep((REV ? p.Y : p.E) + it * kTile, u, row);
    }
    if (LEAN) {  // what the gradient scales their products by
      uint32_t m = kNoMax;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max_finite(m, row * u[j]);
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) atomicMax(REV ? &p.tab[it].mw : &p.tab[it].mu, max_bits(m));
    }
    float bc[8];
    if (REV) {
      float er[8];
      wait_bar(bars + SB_ERR, x & 1, p.err);
      rows8(s + Sm::kErr, er, 1.f);
      float ew = 0.f, vw = 0.f;
      uint32_t dvw[4];
      const uint32_t vv[4] = {vr.x, vr.y, vr.z, vr.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w0 = sg.y * u[2 * j], w1 = sg.y * u[2 * j + 1], d0 = bt * w0, d1 = bt * w1;
        ew = fmaf(er[2 * j], w0, fmaf(er[2 * j + 1], w1, ew));
        const float2 f = unpack_bf16x2(vv[j]);
        vw = fmaf(f.x, d0, fmaf(f.y, d1, vw));
        dvw[j] = pack_bf16x2(d0, d1);
      }
      const int t = c * kC + i;
      p.part[(it * kParts + sl * 4 + qt) * kC + i] = make_float2(ew, vw);
      if (t < sq.len && cols_in)
        *reinterpret_cast<uint4*>(p.dval + (row0 + t) * p.dv + col0) = make_uint4(dvw[0], dvw[1], dvw[2], dvw[3]);
      wait_bar(bars + SB_BC, x & 1, p.err);
      rows8(s + Sm::kBc, bc, sg.x);
    }
    wait_mma();
    {
      float hi[8], lo[8];
      tmem_ld8(tl + 128, hi);
      tmem_ld8(tl + 160, lo);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = fmaf(kLoInv, lo[j], hi[j]);
        X[j] = fmaf(gam, X[j], REV ? fmaf(-in0, y, bc[j]) : y);
      }
    }
  }
  float* to = REV ? p.dstate_in : MODE == kFwdKeep ? p.final_state : p.state_out;
  if (to && i < p.dk && cols_in) {
#pragma unroll
    for (int j = 0; j < 8; ++j) to[(sh * p.dv + col0 + j) * p.dk + i] = X[j] * sg.y;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------------------------- output
constexpr uint32_t kOQ = 0;                  // Q
constexpr uint32_t kOK = kOQ + kTile;        // K; then the masked scores
constexpr uint32_t kOS = kOK + kTile;        // X; then u
constexpr uint32_t kOTab = kOS + kTile;
constexpr uint32_t kOBars = kOTab + 2 * kC * 4 + 32;
constexpr uint32_t kOCol = kOBars + 32;
constexpr uint32_t kOutSmem = kOCol + kColDecays * 4;

// One CTA per (chunk, head), two per SM, so that one's loads and stores run beside the
// other's products.  Bound by memory: 160 KB an item, 336 MB for 2048 items in 64 us, 5.2 TB/s.
__global__ void __launch_bounds__(256, 2) gdr_out_kernel(const __grid_constant__ TcMaps maps, TcParams p) {
  extern __shared__ __align__(1024) unsigned char s[];
  wait_for_previous();
  if (smem_u32(s) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceArg);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, hf = warp >> 2, i = 32 * q + lane;
  const int it = blockIdx.x, slot = it / p.seqs.H, h = it - slot * p.seqs.H;
  const int hk = h / (p.seqs.H / p.seqs.Hk);
  int seq, chunk;
  GdrSeq sq;
  if (!gdr_find(p.seqs, slot, kC, seq, chunk, sq)) return;
  const int t0 = chunk * kC, n = min(kC, sq.len - t0);
  const size_t row0 = ((size_t)sq.row_b * p.seqs.H + h) * p.seqs.T + sq.start + t0;
  const size_t krow0 = ((size_t)sq.row_b * p.seqs.Hk + hk) * p.seqs.T + sq.start + t0;
  float2* gs = reinterpret_cast<float2*>(s + kOTab);
  uint32_t* red = reinterpret_cast<uint32_t*>(gs + kC);
  uint64_t* bars = reinterpret_cast<uint64_t*>(s + kOBars);  // 0: K and X, then u; 1: products; 2: Q
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + kOBars + 24);
  const uint32_t sQ = smem_u32(s + kOQ), sK = smem_u32(s + kOK), sS = smem_u32(s + kOS);
  if (tid == 0) {
    for (int b = 0; b < 3; ++b) mbar_init(bars + b, 1);
    fence_mbar_init();
    load_tile(s + kOQ, &maps.q, (int)krow0, bars + 2);
    mbar_arrive_expect_tx(bars, 2 * kTile);
    bulk_load(s + kOK, p.K16 + ((size_t)slot * p.seqs.Hk + hk) * kTile, kTile, bars);
    bulk_load(s + kOS, p.S + (size_t)it * kTile, kTile, bars);
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  float* cf = reinterpret_cast<float*>(s + kOCol);
  if (tid < kC) gs[tid] = p.tab[it].g[tid];
  column_decays(cf, p.tab[it].g, tid);
  const float ie = pow2_inverse(p.tab[it].all.w), isf = operand_scale(__uint_as_float(p.amax_s[(size_t)seq * p.seqs.H + h])).y;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + 64 * hf;
  wait_bar(bars + 2, 0, p.err);
  const float iq = tile_to_f16<256>(s + kOQ, n, red, tid, 0);
  __syncthreads();
  if (tid == 0) {
    wait_bar(bars, 0, p.err);
    tc_fence_after();
    mma_tile<kAlong, kAlong>(tmem, sQ, sK, false);
    mma_tile<kAlong, kPlainDown>(tmem + 128, sQ, sS, false);
    umma_commit(bars + 1);
  }
  __syncwarp();
  wait_bar(bars + 1, 0, p.err);
  __syncwarp();
  tc_fence_after();
  if (tid == 0) {
    mbar_arrive_expect_tx(bars, kTile);
    bulk_load(s + kOS, p.E + (size_t)it * kTile, kTile, bars);
  }
  __syncwarp();
  const float2 gi = gs[i];
#pragma unroll
  for (int c = 0; c < 2; ++c) {  // Q K^T . G over K
    const int j0 = 64 * hf + 32 * c;
    float a[32], dec[32];
    tmem_ld32(tl + 32 * c, a);
    row_decays<32>(dec, cf, gs, gi, i, q, j0);
    tmem_ld_wait();
#pragma unroll
    for (int jj = 0; jj < 32; ++jj) a[jj] = j0 + jj <= i ? kScoreDown * a[jj] * dec[jj] : 0.f;
#pragma unroll
    for (int c8 = 0; c8 < 4; ++c8)
      *reinterpret_cast<uint4*>(s + kOK + swz16(i, (j0 >> 3) + c8)) =
          make_uint4(pack_f16x2(a[8 * c8], a[8 * c8 + 1]), pack_f16x2(a[8 * c8 + 2], a[8 * c8 + 3]),
                     pack_f16x2(a[8 * c8 + 4], a[8 * c8 + 5]), pack_f16x2(a[8 * c8 + 6], a[8 * c8 + 7]));
  }
  fence_proxy_async_shared();
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    wait_bar(bars, 1, p.err);
    tc_fence_after();
    mma_tile<kAlong, kPlainDown>(tmem, sK, sS, false);
    umma_commit(bars + 1);
  }
  __syncwarp();
  wait_bar(bars + 1, 1, p.err);
  __syncwarp();
  tc_fence_after();
  const float fx = p.scale * iq * isf * exp_diff(gi, make_float2(0.f, 0.f));
  const float fa = p.scale * iq * ie * isf / kScoreDown;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int j0 = 64 * hf + 32 * c;
    if (j0 >= p.dv) continue;
    float a[32], x[32];
    tmem_ld32(tl + 32 * c, a);
    tmem_ld32(tl + 128 + 32 * c, x);
    tmem_ld_wait();
#pragma unroll
    for (int v = 0; v < 4; ++v) {  // by way of Q's place, whole rows to half a warp
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 8 * v + 2 * e;
        w[e] = pack_bf16x2(fmaf(fx, x[j], fa * a[j]), fmaf(fx, x[j + 1], fa * a[j + 1]));
      }
      *reinterpret_cast<uint4*>(s + kOQ + swz16(i, (j0 >> 3) + v)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  store_rows(p.o + row0 * p.dv, s + kOQ, n, p.dv, tid, 256);
  __syncwarp();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---------------------------------------------------------------- gradients
constexpr uint32_t kGBars = 7 * kTile;
constexpr uint32_t kGTab = kGBars + 6 * 8;
constexpr uint32_t kGNext = kGTab + 2 * kC * 4 + 32;
constexpr uint32_t kGCol = (kGNext + sizeof(Item) + 15) / 16 * 16;
constexpr uint32_t kGradSmem = kGCol + kColDecays * 4;
static_assert(kGradSmem <= 232448, "shared memory budget of one CTA");
constexpr int kGradThreads = 512;

// Persistent, one CTA per SM, an item per (chunk, key head); the value heads that
// share it are taken in turn, dq and dk adding up in registers in a fixed order.
// Thread = (row, quarter of the columns).  The next head's or item's tiles are
// loaded as soon as a tile's last product is done.  Measured: 113 us for 1024 items (415 MB,
// 3.7 TB/s; 140 with a CTA per item, whose loads nothing overlapped), bound by the
// chain of its three rounds.  Per head three rounds of products over seven tiles of
// shared memory:
//   dO S, (beta w) S, u D;   dO u^T, (beta w) u^T, Q K^T;   R K, R^T Q, (N + N^T) K
// with R = scale (dO u^T . G) and N = ((beta w) u^T . G) strictly lower, as operands
// scaled by what brings the largest elements of u' and p beta w (known from the scans) to 16,
// as that of dO is: a sum of 128 products stays below 2^15, however far states grew.  The
// first and fourth take S and u in two parts: q.dq, which enters dlog_alpha, is
// then exact to float32; the rest ends in 16-bit gradients.
__global__ void __launch_bounds__(kGradThreads, 1) gdr_grad_tc_kernel(TcParams p) {
  extern __shared__ __align__(1024) unsigned char s[];
  wait_for_previous();
  if (smem_u32(s) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceArg);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, qt = warp >> 2, i = 32 * q + lane, j0 = 32 * qt;
  const int G = p.seqs.H / p.seqs.Hk, units = p.slots * p.seqs.Hk;
  Item* next = reinterpret_cast<Item*>(s + kGNext);
  uint64_t* bars = reinterpret_cast<uint64_t*>(s + kGBars);  // 0: Y and u, 1: dO, S and D, 2: Q and K, 3: products
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + kGBars + 4 * 8);
  float2* gs = reinterpret_cast<float2*>(s + kGTab);
  double* tot = reinterpret_cast<double*>(gs + kC);        // [4]
  // tiles: 0 dO, then N; 1-2 S, then Q and K; 3 beta w; 4-5 u; 6 D, then R
  constexpr uint32_t tO = 0, tS = kTile, tQ = kTile, tK = 2 * kTile, tY = 3 * kTile, tU = 4 * kTile, tD = 6 * kTile;
  constexpr uint32_t kLow = 64;  // of a slice tile's low part
  float* cf = reinterpret_cast<float*>(s + kGCol);  // the columns' decay factors
  if (tid == 0) {
    for (int b = 0; b < 4; ++b) mbar_init(bars + b, 1);
    fence_mbar_init();
    find_unit(p, blockIdx.x, gridDim.x, next);
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + j0;
  const uint32_t s0 = smem_u32(s);
  uint32_t nmma = 0;
  auto wait_mma = [&]() {
    wait_bar(bars + 3, nmma & 1, p.err);
    ++nmma;
    __syncwarp();
    tc_fence_after();
  };
  // loads of (slot, head) item `it`, by thread 0
  auto load_rows = [&](size_t it) {
    mbar_arrive_expect_tx(bars, 3 * kTile);
    bulk_load(s + tY, p.Y + it * kTile, kTile, bars);
    bulk_load(s + tU, p.E + it * 2 * kTile, 2 * kTile, bars);
  };
  auto load_do = [&](size_t it) {  // and D, as soon as N and R have been read
    mbar_arrive_expect_tx(bars + 1, 4 * kTile);
    bulk_load(s + tO, p.dO16 + it * kTile, kTile, bars + 1);
    bulk_load(s + tD, p.D + it * kTile, kTile, bars + 1);
  };
  auto load_s = [&](size_t it) { bulk_load(s + tS, p.S + it * 2 * kTile, 2 * kTile, bars + 1); };
  auto head_of = [&](int unit, int hh) {  // (slot, head) of a unit's head
    const int slot = unit / p.seqs.Hk;
    return (size_t)slot * p.seqs.H + (unit - slot * p.seqs.Hk) * G + hh;
  };
  float xq[32], xk[32];  // dq and dk of this thread's row and columns, over the heads
  Item me = *next;
  if (tid == 0 && me.it < units) {
    load_rows(head_of(me.it, 0));
    load_do(head_of(me.it, 0));
    load_s(head_of(me.it, 0));
  }
  __syncwarp();
  uint32_t par = 0;
  while (me.it < units) {
    __syncthreads();  // (the item has been read)
    if (tid == 511) find_unit(p, me.it + gridDim.x, gridDim.x, next);
    const int unit = me.it, n = me.n;
    const size_t krow0 = me.krow0;
#pragma unroll
    for (int j = 0; j < 32; ++j) xq[j] = xk[j] = 0.f;
    for (int hh = 0; hh < G; ++hh, par ^= 1) {
      const size_t it = head_of(unit, hh), sh = (size_t)me.seq * p.seqs.H + (unit % p.seqs.Hk) * G + hh;
      const size_t row0 = me.row0 + (size_t)hh * p.seqs.T;
      if (tid == 0) {
        wait_bar(bars, par, p.err);
        wait_bar(bars + 1, par, p.err);
        tc_fence_after();
        mma_tile<kAlong, kSlices>(tmem, s0 + tO, s0 + tS, false);
        mma_tile<kAlong, kSlices>(tmem + 128, s0 + tO, s0 + tS + kLow, false);
        mma_tile<kPlain, kSlices>(tmem + 256, s0 + tY, s0 + tS, false);
        mma_tile<kSlices, kPlain>(tmem + 384, s0 + tU, s0 + tD, false);
        umma_commit(bars + 3);
      }
      __syncwarp();
      const Tables& tb = p.tab[it];
      if (tid < kC) gs[tid] = tb.g[tid];
      column_decays(cf, tb.g, tid - 256 < 0 ? kColDecays : tid - 256);
      float* dg = reinterpret_cast<float*>(p.part + (it * kParts + 16) * kC);  // [4][token]
      // factors of products: fo of dO S, fr of dO (eps u')^T, fn of (eps p beta w) (eps u')^T, fs of eps u' D and
      // eps p beta w S, with 1 / p of a row of dk
      const float isf = operand_scale(__uint_as_float(p.amax_s[sh])).y, isr = operand_scale(__uint_as_float(p.amax_d[sh])).y;
      const float ie = pow2_inverse(tb.all.w), ip = pow2_inverse(tb.p[i]), iq = tb.iq, fo = p.scale * tb.id * isf, fr = fo * ie;
      const float fs = isf * isr * ie * ip, fn = -fs * ie, fq = fo * tb.into[i], fu = fs * tb.out[i], fw = -fs * tb.into[i];
      // of R and N as operands (what is below 2^-24 is zero in fp16)
      const float up_r = operand_scale(fmaxf(__uint_as_float(tb.mu), 0x1p-24f)).x;
      const float up_n = up_r * operand_scale(fmaxf(__uint_as_float(tb.mw), 0x1p-24f)).x;
      uint4 qv[4];  // this thread's piece of Q's row
#pragma unroll
      for (int v = 0; v < 4; ++v)
        qv[v] = i < n && j0 < p.dk ? *reinterpret_cast<const uint4*>(p.q + (krow0 + i) * p.dk + j0 + 8 * v)
                                   : make_uint4(0u, 0u, 0u, 0u);
      wait_mma();
      if (tid == 0) {
        mbar_arrive_expect_tx(bars + 2, 2 * kTile);
        bulk_load(s + tQ, p.Q16 + (size_t)unit * kTile, kTile, bars + 2);
        bulk_load(s + tK, p.K16 + (size_t)unit * kTile, kTile, bars + 2);
      }
      __syncwarp();
      // ---- round 1: dq's and dk's parts by the states, q.dq's first part
      float qdot = 0.f;
      {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float a[16], x[16];
          tmem_ld16(tl + 256 + 16 * c, a);
          tmem_ld16(tl + 384 + 16 * c, x);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) xk[16 * c + j] += fmaf(fu, x[j], fw * a[j]);
          tmem_ld16(tl + 16 * c, a);
          tmem_ld16(tl + 128 + 16 * c, x);
          tmem_ld_wait();
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint4 qq = qv[2 * c + v];
            const uint32_t w[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = 8 * v + 2 * e;
              const float y0 = fq * fmaf(kLoInv, x[j], a[j]), y1 = fq * fmaf(kLoInv, x[j + 1], a[j + 1]);
              const float2 f = unpack_bf16x2(w[e]);
              qdot = fmaf(f.x, y0, fmaf(f.y, y1, qdot));
              xq[16 * c + j] += y0;
              xq[16 * c + j + 1] += y1;
            }
          }
        }
      }
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        mma_tile<kAlong, kSlices>(tmem + 128, s0 + tO, s0 + tU + kLow, false);
        mma_tile<kAlong, kSlices>(tmem + 128, s0 + tO, s0 + tU, true);
        mma_tile<kPlain, kSlices>(tmem + 256, s0 + tY, s0 + tU, false);
        wait_bar(bars + 2, par, p.err);
        mma_tile<kAlong, kAlong>(tmem + 384, s0 + tQ, s0 + tK, false);
        umma_commit(bars + 3);
      }
      __syncwarp();
      wait_mma();
      if (tid == 0 && (hh + 1 < G || next->it < units)) load_rows(hh + 1 < G ? it + 1 : head_of(next->it, 0));
      __syncwarp();
      // ---- round 2: R and N as operands; q.dq's second part, the row sums of R . Q K^T
      {
        const float2 gi = gs[i];
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float r[16], a[16], dec[16];
          row_decays<16>(dec, cf, gs, gi, i, q, j0 + 16 * c);
          tmem_ld16(tl + 128 + 16 * c, r);
          tmem_ld16(tl + 384 + 16 * c, a);
          tmem_ld_wait();
#pragma unroll
          for (int jj = 0; jj < 16; ++jj) {
            const int j = j0 + 16 * c + jj;
            r[jj] = j <= i ? r[jj] * dec[jj] : 0.f;
            if (j <= i) sum = fmaf(r[jj], a[jj], sum);
          }
          tmem_ld16(tl + 256 + 16 * c, a);
          tmem_ld_wait();
#pragma unroll
          for (int c8 = 0; c8 < 2; ++c8) {
            uint32_t rr[4], nw[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int jj = 8 * c8 + 2 * e, j = j0 + 16 * c + jj;
              rr[e] = pack_f16x2(up_r * r[jj], up_r * r[jj + 1]);
              nw[e] = pack_f16x2(j < i ? up_n * dec[jj] * a[jj] : 0.f, j + 1 < i ? up_n * dec[jj + 1] * a[jj + 1] : 0.f);
            }
            const uint32_t at = swz16(i, 4 * qt + 2 * c + c8);
            *reinterpret_cast<uint4*>(s + tD + at) = make_uint4(rr[0], rr[1], rr[2], rr[3]);
            *reinterpret_cast<uint4*>(s + tO + at) = make_uint4(nw[0], nw[1], nw[2], nw[3]);
          }
        }
        dg[qt * kC + i] = fmaf(fr * iq, sum, qdot);
      }
      fence_proxy_async_shared();
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        mma_tile<kAlong, kDown>(tmem + 128, s0 + tD, s0 + tK, false);  // R K
        mma_tile<kDown, kDown>(tmem + 256, s0 + tD, s0 + tQ, false);   // R^T Q
        mma_tile<kAlong, kDown>(tmem + 384, s0 + tO, s0 + tK, false);  // N K
        mma_tile<kDown, kDown>(tmem + 384, s0 + tO, s0 + tK, true);    // N^T K
        umma_commit(bars + 3);
      }
      __syncwarp();
      // ---- the gates' gradients: sums over the slices, the suffix sum over the chunk
      if (warp >= 12) {
        const int t = tid - 384;
        const float la = t < n ? p.log_alpha[row0 + t] : 0.f;
        float ew = 0.f, vw = 0.f;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float2 f = p.part[(it * kParts + x) * kC + t];
          ew += f.x;
          vw += f.y;
        }
        double y = t < n ? (double)(((dg[t] + dg[kC + t]) + (dg[2 * kC + t] + dg[3 * kC + t])) - vw) : 0.0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double z = __shfl_down_sync(0xffffffffu, y, o);
          if (lane + o < 32) y += z;
        }
        if (lane == 0) tot[q] = y;
        float bsum = p.bnd[it * kBnd + lane] + p.bnd[it * kBnd + 32 + lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bsum += __shfl_xor_sync(0xffffffffu, bsum, o);
        named_bar_sync(1, kC);
        for (int w = q + 1; w < 4; ++w) y += tot[w];
        if (t < n) {
          p.dlog_alpha[row0 + t] = gdr_forgets(la) ? 0.f : (float)(y + (double)bsum);
          p.dbeta[row0 + t] = ew;
        }
      }
      wait_mma();
      if (tid == 0 && (hh + 1 < G || next->it < units)) load_do(hh + 1 < G ? it + 1 : head_of(next->it, 0));
      __syncwarp();
      // ---- round 3
      {
        const float f0 = fr * pow2_inverse(up_r), f1 = f0 * iq * ip, f2 = fn * pow2_inverse(up_n);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float a[16], x[16], y[16];
          tmem_ld16(tl + 128 + 16 * c, y);
          tmem_ld16(tl + 256 + 16 * c, a);
          tmem_ld16(tl + 384 + 16 * c, x);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            xk[16 * c + j] += fmaf(f1, a[j], f2 * x[j]);
            xq[16 * c + j] = fmaf(f0, y[j], xq[16 * c + j]);
          }
        }
      }
      if (hh + 1 == G) {  // the gradients leave by way of Q's and K's places, whole rows to a warp
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const uint32_t at = swz16(i, 4 * qt + v);
          *reinterpret_cast<uint4*>(s + tQ + at) =
              make_uint4(pack_bf16x2(xq[8 * v], xq[8 * v + 1]), pack_bf16x2(xq[8 * v + 2], xq[8 * v + 3]),
                         pack_bf16x2(xq[8 * v + 4], xq[8 * v + 5]), pack_bf16x2(xq[8 * v + 6], xq[8 * v + 7]));
          *reinterpret_cast<uint4*>(s + tK + at) =
              make_uint4(pack_bf16x2(xk[8 * v], xk[8 * v + 1]), pack_bf16x2(xk[8 * v + 2], xk[8 * v + 3]),
                         pack_bf16x2(xk[8 * v + 4], xk[8 * v + 5]), pack_bf16x2(xk[8 * v + 6], xk[8 * v + 7]));
        }
        __syncthreads();
        store_rows(p.dq + krow0 * p.dk, s + tQ, n, p.dk, tid, kGradThreads);
        store_rows(p.dkey + krow0 * p.dk, s + tK, n, p.dk, tid, kGradThreads);
      }
      fence_proxy_async_shared();
      tc_fence_before();
      __syncthreads();  // the next head's tiles and tables
      tc_fence_after();
      if (tid == 0 && (hh + 1 < G || next->it < units)) load_s(hh + 1 < G ? it + 1 : head_of(next->it, 0));
      __syncwarp();
    }
    me = *next;
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- host side
struct Plan {
  size_t W, U, K16, S, E, tab, amax, amax_bytes;
  size_t Q16, dO16, Wd, w0, Bc, D, Y, fin, part, bnd;
  size_t total;
  int slots;
};
Plan plan_of(const GdrArgs& a, bool bwd) {
  Plan p{};
  const size_t slots = gdr_slots(a, kC), items = slots * a.H, rows = items * kC * kC * 4;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at = align_up(at + bytes, 1024);
    return x;
  };
  p.slots = (int)slots;
  const int parts = bwd ? 2 : 1;
  p.W = take(items * 2 * kTile);
  p.U = take(rows);
  p.K16 = take(slots * a.Hk * kTile);
  p.S = take(items * parts * kTile);
  p.E = take(items * parts * kTile);
  p.tab = take(items * sizeof(Tables));
  p.amax_bytes = (size_t)2 * gdr_sequences(a) * a.H * 4;
  p.amax = take(p.amax_bytes);
  if (bwd) {
    p.Q16 = take(slots * a.Hk * kTile);
    p.dO16 = take(items * kTile);
    p.Wd = take(items * 2 * kTile);
    p.w0 = take(rows);
    p.Bc = take(rows);
    p.D = take(items * kTile);
    p.Y = take(items * kTile);
    p.fin = take((size_t)gdr_sequences(a) * a.H * a.dv * a.dk * 4);
    p.part = take(items * kParts * kC * sizeof(float2));
    p.bnd = take(items * kBnd * 4);
  }
  p.total = at;
  return p;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

TcParams params_of(const GdrArgs& a, const Plan& pl, bool bwd) {
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  TcParams p{};
  p.seqs = GdrSeqs{a.n_seqs ? a.seq_starts : nullptr, gdr_sequences(a), a.T, a.H, a.Hk};
  p.dk = a.dk;
  p.dv = a.dv;
  p.slots = pl.slots;
  p.scale = a.scale;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.dout = static_cast<const __nv_bfloat16*>(a.dout);
  p.log_alpha = a.log_alpha;
  p.beta = a.beta;
  p.state_in = a.state_in;
  p.dstate_out = a.dstate_out;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.state_out = a.state_out;
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dkey = static_cast<__nv_bfloat16*>(a.dkey);
  p.dval = static_cast<__nv_bfloat16*>(a.dval);
  p.dlog_alpha = a.dlog_alpha;
  p.dbeta = a.dbeta;
  p.dstate_in = a.dstate_in;
  p.W = ws + pl.W;
  p.U = reinterpret_cast<float*>(ws + pl.U);
  p.K16 = ws + pl.K16;
  p.S = ws + pl.S;
  p.E = ws + pl.E;
  p.tab = reinterpret_cast<Tables*>(ws + pl.tab);
  p.amax_s = reinterpret_cast<unsigned*>(ws + pl.amax);
  p.amax_d = p.amax_s + (size_t)gdr_sequences(a) * a.H;
  if (bwd) {
    p.Q16 = ws + pl.Q16;
    p.dO16 = ws + pl.dO16;
    p.Wd = ws + pl.Wd;
    p.w0 = reinterpret_cast<float*>(ws + pl.w0);
    p.Bc = reinterpret_cast<float*>(ws + pl.Bc);
    p.D = ws + pl.D;
    p.Y = ws + pl.Y;
    p.final_state = reinterpret_cast<float*>(ws + pl.fin);
    p.part = reinterpret_cast<float2*>(ws + pl.part);
    p.bnd = reinterpret_cast<float*>(ws + pl.bnd);
  }
  p.err = a.err;
  return p;
}

// a kernel that begins with wait_for_previous()
template <typename... P, typename... A>
ll_status launch_next(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                      const A&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = &at;
  c.numAttrs = 1;
  LL_CUDA_OK(cudaLaunchKernelEx(&c, kernel, args...));
  return LL_OK;
}
template <int MODE> ll_status scan(const GdrArgs& a, const TcParams& p, int slices) {
  LL_CUDA_OK(cudaFuncSetAttribute(gdr_scan_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)ScanSm<MODE>::kBytes));
  return launch_next(gdr_scan_kernel<MODE>, (unsigned)(gdr_sequences(a) * a.H * slices), kScanThreads,
                     ScanSm<MODE>::kBytes, a.stream, p, slices);
}
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  auto f = fn.load(std::memory_order_acquire);
  if (!f) {  // (threads may look it up at once)
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &qr) !=
            cudaSuccess ||
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
bool maps_of(const GdrArgs& a, TcMaps* m) {
  const uint64_t rows = (uint64_t)a.B * a.H * a.T, krows = (uint64_t)a.B * a.Hk * a.T;
  return make_map(&m->q, a.q, krows, a.dk) && make_map(&m->k, a.k, krows, a.dk) && make_map(&m->v, a.v, rows, a.dv) &&
         make_map(&m->dout, a.dout ? a.dout : a.v, rows, a.dv);
}
ll_status prep(const GdrArgs& a, const TcMaps& m, const TcParams& p, const Plan& pl, bool bwd) {
  const int items = pl.slots * a.H, sms = sm_count();
  if (sms == 0) return LL_ERR_CUDA;
  auto kernel = bwd ? gdr_prep_bwd_kernel : gdr_prep_fwd_kernel;
  LL_CUDA_OK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PrepSm::kBytes));
  LL_CUDA_OK(cudaMemsetAsync(p.amax_s, 0, pl.amax_bytes, a.stream));
  kernel<<<std::min(items, sms), kPrepThreads, PrepSm::kBytes, a.stream>>>(m, p);
  LL_CUDA_OK(cudaGetLastError());
  return LL_OK;
}

}  // namespace

// bf16 io, head sizes of 64 and 128; rows are 32-bit coordinates of the copies
static bool tc_formats(const GdrArgs& a) {
  return a.io == LL_BF16 && a.dk >= 64 && a.dv >= 64 && (long long)a.B * a.H * a.T <= (1ll << 31) - 1 - kC;
}
// Which of the two ways is faster follows from both measured, in us, for 4 to
// 1024 (sequence, head) pairs of 1 to 1024 tokens and for packed batches of 512
// to 8192 tokens.  Token by token a forward takes 4 plus the larger of its longest
// sequence's tokens (0.12 each at d_k = 128, 0.095 at 64, 1.6 times that once the
// rows of all states are 4096 and more and blocks share an SM) and of all of them
// (0.0058 a token and head at 128 x 128, less in proportion to the state); in
// chunks it takes three launches (34 in all, however small), or 0.18 an item and 0.06 a
// state (0.15 and 0.05 with a side of 64).  For 16 heads of one sequence (128 x 128,
// token by token / in chunks): 19.5 / 34.8 at 128 tokens, 35.1 / 37.1 at 256, 50.8 / 38.3 at
// 384; for 1024 heads: 202 / 257 at 32 tokens, 363 / 262 at 64.  Only the device
// knows the lengths of packed sequences: their mean is T / n, the longest is
// taken for twice that.  The choice is the slower one, by 10 % or more, in 12 of
// 451 shapes measured, by 1.53 times at most.  None of these is a packed batch of few
// heads with nearly all of its tokens in one sequence, which goes token by token and is
// one long chain: 64 sequences of 4096 tokens on one head 605 us, in chunks 101 (of even
// lengths 38 and 49), 256 of them on two heads 823 and 216 (74 and 163).  Either choice is
// the slower one for some lengths; a caller who knows of such a sequence can pass it alone.
bool gdr_tc_fwd_use(const GdrArgs& a) {
  if (!tc_formats(a)) return false;
  const double seqs = gdr_sequences(a), states = seqs * a.H, wide = a.dk * a.dv / 4096.;
  const double mean = a.n_seqs ? std::ceil(a.T / seqs) : a.T, longest = a.n_seqs > 1 ? std::min<double>(a.T, 2 * mean) : a.T;
  const double token = (a.dk > 64 ? 0.12 : 0.095) * (!a.n_seqs && states * a.dv >= 4096 ? 1.6 : 1.);
  const double by_token = 4 + std::max(token * longest, 0.00145 * wide * mean * states);
  const double items = states * std::ceil(mean / kC);
  const double in_chunks = std::max(34., 18 + (wide == 4 ? 0.18 : 0.15) * items + (wide == 4 ? 0.06 : 0.05) * states);
  return in_chunks < by_token;
}
// The gradient: token by token it takes a launch over both recurrences and one over
// chunks of 64.  At 128 x 128 the tensor cores are the faster at every length but a
// token of many heads (16 heads: 78 / 58 us at 1 token, 82 / 58 at 16; 256 heads: 174 / 179 at 1,
// 207 / 179 at 16; 8192 heads: 7008 / 4417 at 16, 11323 / 4504 at 64); the bound of 16 is for the workspace
// too, whose items are padded to 128 tokens (8192 heads of 16 tokens: 1.2 / 5.8 GB).  With one side of 64 they are from 64 tokens on (64 x 128, 256 heads:
// 168 / 181 at 32, 219 / 182 at 64; 128 x 64, 16 heads: 52 / 59 at 32, 59 / 59 at 64), with two from
// 128 (16 heads: 52 / 60 at 128, 66 / 64 at 256; 64 heads: 68 / 70 at 128, 111 / 90 at 192; 256 heads:
// 244 / 180 at 128).
bool gdr_tc_bwd_use(const GdrArgs& a) {
  const int mean = a.n_seqs ? (a.T + a.n_seqs - 1) / a.n_seqs : a.T;
  return tc_formats(a) && mean >= (a.dk * a.dv > 64 * 128 ? 16 : a.dk * a.dv > 64 * 64 ? 64 : 128);
}
size_t gdr_tc_fwd_workspace(const GdrArgs& a) { return plan_of(a, false).total; }
size_t gdr_tc_bwd_workspace(const GdrArgs& a) { return plan_of(a, true).total; }

ll_status gdr_tc_fwd_launch(const GdrArgs& a) {
  const Plan pl = plan_of(a, false);
  const TcParams p = params_of(a, pl, false);
  TcMaps m;
  if (!maps_of(a, &m)) return LL_ERR_CUDA;
  ll_status st = prep(a, m, p, pl, false);
  if (st == LL_OK) st = scan<kFwd>(a, p, a.dv / kSlice);
  if (st != LL_OK) return st;
  LL_CUDA_OK(cudaFuncSetAttribute(gdr_out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kOutSmem));
  return launch_next(gdr_out_kernel, (unsigned)(pl.slots * a.H), 256, kOutSmem, a.stream, m, p);
}

ll_status gdr_tc_bwd_launch(const GdrArgs& a) {
  const Plan pl = plan_of(a, true);
  const TcParams p = params_of(a, pl, true);
  TcMaps m;
  if (!maps_of(a, &m)) return LL_ERR_CUDA;
  ll_status st = prep(a, m, p, pl, true);
  // all slices, so that the columns behind a d_v of 64 are zeros: they are summed over
  if (st == LL_OK) st = scan<kFwdKeep>(a, p, kC / kSlice);
  if (st == LL_OK) st = scan<kRev>(a, p, kC / kSlice);
  if (st != LL_OK) return st;
  LL_CUDA_OK(cudaFuncSetAttribute(gdr_grad_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGradSmem));
  const int sms = sm_count();
  if (sms == 0) return LL_ERR_CUDA;
  return launch_next(gdr_grad_tc_kernel, (unsigned)std::min(pl.slots * a.Hk, sms), kGradThreads, kGradSmem, a.stream, p);
}

}  // namespace llattn

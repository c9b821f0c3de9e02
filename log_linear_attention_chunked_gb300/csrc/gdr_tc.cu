// The gated delta rule's forward on the 5th-generation tensor cores: bf16 io,
// head sizes 64 and 128, 128-token chunks.
//
// Chunk (g = running log decay inside it, G_ij = exp(g_i - g_j) for j <= i, S0
// the state before it, X = S0^T):
//   T = (I + diag(beta) SL(K K^T . G))^-1      U = T diag(beta) V
//   W = T diag(beta exp(g)) K                  u = U - W X     (the rows written)
//   O = scale (diag(exp(g)) Q X + (Q K^T . G) u)
//   X <- exp(g_C) X + K^T diag(exp(g_C - g)) u
// Three kernels: the preparation (U, W; parallel over chunks), the scan (u and
// the states; sequential over a sequence's chunks, parallel over heads and
// slices of 32 d_v columns) and the output (parallel over chunks).  The states
// are float32 results: the first two keep float32 accuracy by split operands
// (gdr_tc.cuh); the output rounds X, u and the masked scores to bf16 once each,
// as its own result is.
#include <algorithm>

#include "gdr_tc.cuh"

namespace llattn {

namespace {

using namespace gdrtc;

// per (chunk, head): decay tables
struct Tables {
  float2 g[kC];    // running log decay
  float into[kC];  // exp(g_t)
  float out[kC];   // exp(g_C - g_t)
};

struct TcParams {
  GdrSeqs seqs;
  int dk, dv, slots;
  float scale;
  const __nv_bfloat16 *q, *k, *v;
  const float *log_alpha, *beta, *state_in;
  __nv_bfloat16* o;
  float* state_out;
  // workspace, per (slot, head) unless said otherwise
  unsigned char* W;      // two fp16 tiles
  float* U;              // [slice of 32][piece of 4][token][4]
  unsigned char* K16;    // per (slot, key head): K in fp16
  unsigned char* S;      // X before the chunk, bf16 tile [d_k][d_v]
  unsigned char* E;      // u, bf16 tile [token][d_v]
  Tables* tab;
  unsigned* amax;        // [sequence, head]: largest |v|, as bits
  unsigned* err;
};

// ---------------------------------------------------------------- preparation
constexpr uint32_t kPK = 0;                     // K
constexpr uint32_t kPV = kPK + kTile;           // V
constexpr uint32_t kPT = kPV + kTile;           // T's blocks, float32
constexpr uint32_t kPR = kPT + kBlocksB;        // L's blocks; then three parts of T diag(..); then W
constexpr uint32_t kPTab = kPR + 3 * kTile;
constexpr uint32_t kPBars = kPTab + (2 + 1 + 1) * kC * 4 + 32;
constexpr uint32_t kPrepSmem = kPBars + 24;
static_assert(kPR % 1024 == 0 && kPBars % 8 == 0, "tile alignment");
static_assert(kPrepSmem <= 232448, "shared memory budget of one CTA");

// Persistent, one CTA per SM.  T in float32 on the CUDA cores; T diag(beta) and
// T diag(beta exp(g)) as three bf16 parts, so that U and W (three products
// each: V and K are bf16 already) have float32 accuracy.
__global__ void __launch_bounds__(256, 1) gdr_prep_kernel(TcParams p) {
  extern __shared__ __align__(1024) unsigned char s[];
  if (smem_u32(s) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceArg);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, hf = warp >> 2;
  const int i = 32 * q + lane;  // this thread's row (TMEM lane), columns 64 hf ..
  float2* gs = reinterpret_cast<float2*>(s + kPTab);
  float* bs = reinterpret_cast<float*>(gs + kC);
  float* es = bs + kC;
  double* tot = reinterpret_cast<double*>(es + kC);
  uint64_t* bar = reinterpret_cast<uint64_t*>(s + kPBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + kPBars + 8);
  float* Lp = reinterpret_cast<float*>(s + kPR);
  float* Tp = reinterpret_cast<float*>(s + kPT);
  const uint32_t sK = smem_u32(s + kPK), sV = smem_u32(s + kPV), sR = smem_u32(s + kPR);
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
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
  const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
  uint32_t nmma = 0;
  auto wait_mma = [&]() {
    wait_bar(bar, nmma & 1, p.err);
    ++nmma;
    __syncwarp();
    tc_fence_after();
  };

  const int items = p.slots * p.seqs.H, G = p.seqs.H / p.seqs.Hk;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int slot = it / p.seqs.H, h = it - slot * p.seqs.H, hk = h / G;
    int seq, chunk;
    GdrSeq sq;
    if (!gdr_find(p.seqs, slot, kC, seq, chunk, sq)) continue;
    const int t0 = chunk * kC, n = min(kC, sq.len - t0);
    const size_t row0 = ((size_t)sq.row_b * p.seqs.H + h) * p.seqs.T + sq.start + t0;
    const size_t krow0 = ((size_t)sq.row_b * p.seqs.Hk + hk) * p.seqs.T + sq.start + t0;
    if (tid == 0) bulk_wait_read0();  // the item before has left shared memory
    __syncthreads();
    load_tile(s + kPK, p.k + krow0 * p.dk, n, p.dk, tid, 256);
    cp_async_commit();
    load_tile(s + kPV, p.v + row0 * p.dv, n, p.dv, tid, 256);
    cp_async_commit();
    if (tid < kC) bs[tid] = tid < n ? p.beta[row0 + tid] : 0.f;
    chunk_decays(p.log_alpha + row0, n, gs, tot, tid);
    const float2 gi = gs[i], gC = gs[kC - 1];
    const float2 zero = make_float2(0.f, 0.f);
    if (hf == 0) {
      const float in = exp_diff(gi, zero);
      es[i] = in;
      Tables& tb = p.tab[it];
      tb.g[i] = gi;
      tb.into[i] = in;
      tb.out[i] = exp_diff(gC, gi);
    }
    cp_async_wait<1>();
    fence_proxy_async_shared();
    __syncthreads();
    // ---- K K^T -> 0
    if (tid == 0) {
      tc_fence_after();
      mma_tile(tmem, sK, false, sK, false, false);
      umma_commit(bar);
    }
    wait_mma();
    // L_ij = beta_i (k_i . k_j) G_ij, j < i
    {
      const float bt = bs[i];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j0 = 64 * hf + 32 * c;
        if (j0 > 32 * q + 31) continue;  // (warp-uniform) above the diagonal
        float kk[32];
        tmem_ld32(tl + j0, kk);
        tmem_ld_wait();
#pragma unroll
        for (int jj = 0; jj < 32; ++jj) kk[jj] = j0 + jj < i ? bt * kk[jj] * exp_diff(gi, gs[j0 + jj]) : 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int J = (j0 >> 4) + b, I = i >> 4;
          if (J <= I) {
            float4* dst = reinterpret_cast<float4*>(Lp + blk(I, J) + (i & 15) * kBS);
#pragma unroll
            for (int v = 0; v < 4; ++v)
              dst[v] = make_float4(kk[16 * b + 4 * v], kk[16 * b + 4 * v + 1], kk[16 * b + 4 * v + 2],
                                   kk[16 * b + 4 * v + 3]);
          }
        }
      }
    }
    cp_async_wait<0>();  // V, for the barriers below
    __syncthreads();
    tri_inverse(Lp, Tp, tid);
    // the largest |v| of the sequence and head
    {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(s + kPV + swz16(tid >> 1, 8 * (tid & 1) + c));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) atomicMax(p.amax + (size_t)seq * p.seqs.H + h, m << 16);
    }
    // ---- U = T diag(beta) V -> 128, then W = T diag(beta exp(g)) K -> 256
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        const int I = i >> 4, J = 4 * hf + jb;
        float t[16];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float4 x4 = make_float4(0.f, 0.f, 0.f, 0.f);
          if (J <= I) x4 = *reinterpret_cast<const float4*>(Tp + blk(I, J) + (i & 15) * kBS + 4 * v);
          t[4 * v] = x4.x;
          t[4 * v + 1] = x4.y;
          t[4 * v + 2] = x4.z;
          t[4 * v + 3] = x4.w;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int j = 16 * J + e;
          t[e] *= pass == 0 ? bs[j] : bs[j] * es[j];
        }
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = take_bf16x2(t[2 * e], t[2 * e + 1]);
          unsigned char* d = s + kPR + part * kTile;
          *reinterpret_cast<uint4*>(d + swz16(i, 2 * J)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(d + swz16(i, 2 * J + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      fence_proxy_async_shared();
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        const uint32_t d = tmem + 128 + 128 * pass, b = pass == 0 ? sV : sK;
        mma_tile(d, sR + 2 * kTile, false, b, true, false);
        mma_tile(d, sR + kTile, false, b, true, true);
        mma_tile(d, sR, false, b, true, true);
        umma_commit(bar);
      }
      wait_mma();
    }
    // ---- U out, W as two fp16 tiles (over T's parts), K as fp16 in place
    {
      float* ug = p.U + (size_t)it * kC * kC;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j0 = 64 * hf + 32 * c;
        float u[32], w[32];
        tmem_ld32(tl + 128 + j0, u);
        tmem_ld32(tl + 256 + j0, w);
        tmem_ld_wait();
        float4* ud = reinterpret_cast<float4*>(ug) + (size_t)(j0 >> 5) * 8 * kC + i;
#pragma unroll
        for (int v = 0; v < 8; ++v) ud[v * kC] = make_float4(u[4 * v], u[4 * v + 1], u[4 * v + 2], u[4 * v + 3]);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = part == 0 ? take_f16x2(w[8 * c8 + 2 * e], w[8 * c8 + 2 * e + 1])
                               : pack_f16x2(w[8 * c8 + 2 * e], w[8 * c8 + 2 * e + 1]);
            *reinterpret_cast<uint4*>(s + kPR + part * kTile + swz16(i, (j0 >> 3) + c8)) =
                make_uint4(x[0], x[1], x[2], x[3]);
          }
      }
      if (h % G == 0) {
#pragma unroll
        for (int c8 = 0; c8 < 8; ++c8) {
          uint4* at = reinterpret_cast<uint4*>(s + kPK + swz16(i, 8 * hf + c8));
          uint4 v = *at;
          uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_bf16x2(w[e]);
            w[e] = pack_f16x2(f.x, f.y);
          }
          *at = v;
        }
      }
    }
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      bulk_store(p.W + (size_t)it * 2 * kTile, s + kPR, 2 * kTile);
      if (h % G == 0) bulk_store(p.K16 + ((size_t)slot * p.seqs.Hk + hk) * kTile, s + kPK, kTile);
      bulk_commit();
    }
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
constexpr uint32_t kSW = 0;                  // W of two chunks (two fp16 parts each)
constexpr uint32_t kSK = kSW + 4 * kTile;    // K of two chunks (fp16)
constexpr uint32_t kSX = kSK + 2 * kTile;    // X: [d_k][high 32 | low 32] fp16
constexpr uint32_t kSE = kSX + kHalf;        // exp(g_C - g) u: [token][high 32 | low 32]
constexpr uint32_t kSBars = kSE + kHalf;
constexpr uint32_t kSRed = kSBars + 8 * 8;
constexpr uint32_t kScanSmem = kSRed + 64;
static_assert(kScanSmem <= 232448, "shared memory budget of one CTA");
enum ScanBar : int { SB_W0 = 0, SB_W1, SB_K0, SB_K1, SB_MMA, kScanBars };

// One CTA per (32 d_v columns, head, sequence); thread = (TMEM lane, half of the
// columns), the lane a token of the chunk or a d_k row of X in turn.  X stays
// in float32 registers; per chunk two rounds of products, W [Xh | Xl] and
// K^T [uh | ul] (the parts side by side as N = 64: the 128-row operand, which
// shared memory feeds at 128 bytes a cycle, is read once for both).
__global__ void __launch_bounds__(256, 1) gdr_scan_kernel(TcParams p, int slices) {
  extern __shared__ __align__(1024) unsigned char s[];
  if (smem_u32(s) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrDeviceArg);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, hf = warp >> 2, i = 32 * q + lane;
  const int sl = blockIdx.x % slices, h = (blockIdx.x / slices) % p.seqs.H, seq = blockIdx.x / slices / p.seqs.H;
  GdrSeq sq;
  if (!gdr_seq(p.seqs, seq, sq)) {
    if (tid == 0) raise_error(p.err, kErrDeviceArg);
    return;
  }
  const int hk = h / (p.seqs.H / p.seqs.Hk);
  const int col0 = kSlice * sl + 16 * hf;  // this thread's first d_v column
  const int Nc = (sq.len + kC - 1) / kC;
  const int base = gdr_slot_base(p.seqs, seq, sq.start, kC);
  const size_t st0 = ((size_t)seq * p.seqs.H + h) * p.dv;
  float X[16];
#pragma unroll
  for (int j = 0; j < 16; ++j)
    X[j] = p.state_in && i < p.dk && col0 + j < p.dv ? p.state_in[(st0 + col0 + j) * p.dk + i] : 0.f;

  uint64_t* bars = reinterpret_cast<uint64_t*>(s + kSBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + kSBars + kScanBars * 8);
  uint32_t* red = reinterpret_cast<uint32_t*>(s + kSRed);
  auto item = [&](int c) { return (size_t)(base + c) * p.seqs.H + h; };
  auto load_w = [&](int c) {
    mbar_arrive_expect_tx(bars + SB_W0 + (c & 1), 2 * kTile);
    bulk_load(s + kSW + (c & 1) * 2 * kTile, p.W + item(c) * 2 * kTile, 2 * kTile, bars + SB_W0 + (c & 1));
  };
  auto load_k = [&](int c) {
    mbar_arrive_expect_tx(bars + SB_K0 + (c & 1), kTile);
    bulk_load(s + kSK + (c & 1) * kTile, p.K16 + ((size_t)(base + c) * p.seqs.Hk + hk) * kTile, kTile,
              bars + SB_K0 + (c & 1));
  };
  if (tid == 0) {
    for (int b = 0; b < kScanBars; ++b) mbar_init(bars + b, 1);
    fence_mbar_init();
    for (int c = 0; c < 2 && c < Nc; ++c) {
      load_w(c);
      load_k(c);
    }
  }
  uint32_t am = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) am = max(am, __float_as_uint(fabsf(X[j])));
  am = __reduce_max_sync(0xffffffffu, am);
  if (lane == 0) red[warp] = am;
  if (warp == 0) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  am = Nc ? p.amax[(size_t)seq * p.seqs.H + h] : 0u;
#pragma unroll
  for (int w = 0; w < 8; ++w) am = max(am, red[w]);
  const float2 sg = operand_scale(__uint_as_float(am));
#pragma unroll
  for (int j = 0; j < 16; ++j) X[j] *= sg.x;

  const uint32_t tmem = *tmem_slot;
  const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + 16 * hf;
  const uint32_t sX = smem_u32(s + kSX), sE = smem_u32(s + kSE);
  constexpr uint32_t idW = idesc(false, 64, false, true), idK = idesc(false, 64, true, true);
  uint32_t nmma = 0;
  auto wait_mma = [&]() {
    wait_bar(bars + SB_MMA, nmma & 1, p.err);
    ++nmma;
    __syncwarp();
    tc_fence_after();
  };
  // x (16 columns of row i) as high and low fp16 parts of a [row][32 | 32] tile
  auto put = [&](unsigned char* tile, float* x) {
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = part == 0 ? take_f16x2(x[8 * c + 2 * e], x[8 * c + 2 * e + 1])
                           : pack_f16x2(x[8 * c + 2 * e], x[8 * c + 2 * e + 1]);
        *reinterpret_cast<uint4*>(tile + swz16(i, 4 * part + 2 * hf + c)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
  };
  // x times f, rounded to bf16, into row i of a workspace tile
  auto keep = [&](unsigned char* tile, const float* x, float f) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(f * x[8 * c + 2 * e], f * x[8 * c + 2 * e + 1]);
      *reinterpret_cast<uint4*>(tile + swz16(i, (col0 >> 3) + c)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };

  float4 un[4];
  float out_n = 0.f, gam_n = 0.f;
  auto fetch = [&](int c) {
    const float4* ug = reinterpret_cast<const float4*>(p.U) + item(c) * (kC * kC / 4) + (size_t)(sl * 8 + 4 * hf) * kC + i;
#pragma unroll
    for (int v = 0; v < 4; ++v) un[v] = ug[v * kC];
    const Tables& tb = p.tab[item(c)];
    out_n = tb.out[i];
    gam_n = tb.into[kC - 1];
  };
  if (Nc) fetch(0);
  for (int c = 0; c < Nc; ++c) {
    const int b = c & 1;
    // ---- W X
    {
      float x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = X[j];
      put(s + kSX, x);
    }
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      wait_bar(bars + SB_W0 + b, (c >> 1) & 1, p.err);
      tc_fence_after();
      const uint32_t w = smem_u32(s + kSW + b * 2 * kTile);
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_bf16(tmem + 64 * part, desc_k(w + part * kTile, kk), desc_mn(sX, kk), idW, kk > 0);
      umma_commit(bars + SB_MMA);
    }
    keep(p.S + item(c) * kTile, X, sg.y);  // (while the products run)
    float u[16];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      u[4 * v] = sg.x * un[v].x;
      u[4 * v + 1] = sg.x * un[v].y;
      u[4 * v + 2] = sg.x * un[v].z;
      u[4 * v + 3] = sg.x * un[v].w;
    }
    const float fo = out_n, gam = gam_n;
    if (c + 1 < Nc) fetch(c + 1);
    wait_mma();
    if (tid == 0 && c + 2 < Nc) load_w(c + 2);
    {
      float hh[16], hl[16], lh[16];
      tmem_ld16(tl, hh);
      tmem_ld16(tl + 32, hl);
      tmem_ld16(tl + 64, lh);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) u[j] -= fmaf(kLoInv, hl[j] + lh[j], hh[j]);
    }
    // ---- K^T (exp(g_C - g) u)
    {
      float x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = fo * u[j];
      put(s + kSE, x);
    }
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      wait_bar(bars + SB_K0 + b, (c >> 1) & 1, p.err);
      tc_fence_after();
      const uint32_t k = smem_u32(s + kSK + b * kTile);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) umma_bf16(tmem + 128, desc_mn(k, kk), desc_mn(sE, kk), idK, kk > 0);
      umma_commit(bars + SB_MMA);
    }
    keep(p.E + item(c) * kTile, u, sg.y);
    wait_mma();
    if (tid == 0 && c + 2 < Nc) load_k(c + 2);
    {
      float hi[16], lo[16];
      tmem_ld16(tl + 128, hi);
      tmem_ld16(tl + 160, lo);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) X[j] = fmaf(gam, X[j], fmaf(kLoInv, lo[j], hi[j]));
    }
  }
  if (p.state_out) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (i < p.dk && col0 + j < p.dv) p.state_out[(st0 + col0 + j) * p.dk + i] = X[j] * sg.y;
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
constexpr uint32_t kOS = kOK + kTile;        // X
constexpr uint32_t kOE = kOS + kTile;        // u
constexpr uint32_t kOTab = kOE + kTile;
constexpr uint32_t kOBars = kOTab + 2 * kC * 4;
constexpr uint32_t kOutSmem = kOBars + 24;

__global__ void __launch_bounds__(256, 1) gdr_out_kernel(TcParams p) {
  extern __shared__ __align__(1024) unsigned char s[];
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
  uint64_t* bars = reinterpret_cast<uint64_t*>(s + kOBars);  // 0: X and u, 1: products
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s + kOBars + 16);
  const uint32_t sQ = smem_u32(s + kOQ), sK = smem_u32(s + kOK), sS = smem_u32(s + kOS), sE = smem_u32(s + kOE);
  if (tid == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(bars, 2 * kTile);
    bulk_load(s + kOS, p.S + (size_t)it * kTile, kTile, bars);
    bulk_load(s + kOE, p.E + (size_t)it * kTile, kTile, bars);
  }
  load_tile(s + kOQ, p.q + krow0 * p.dk, n, p.dk, tid, 256);
  load_tile(s + kOK, p.k + krow0 * p.dk, n, p.dk, tid, 256);
  cp_async_commit();
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid < kC) gs[tid] = p.tab[it].g[tid];
  cp_async_wait<0>();
  fence_proxy_async_shared();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
  if (tid == 0) {
    mma_tile(tmem, sQ, false, sK, false, false);
    umma_commit(bars + 1);
    wait_bar(bars, 0, p.err);
    mma_tile(tmem + 128, sQ, false, sS, true, false);  // Q X
  }
  __syncwarp();
  wait_bar(bars + 1, 0, p.err);
  __syncwarp();
  tc_fence_after();
  const float2 gi = gs[i];
#pragma unroll
  for (int c = 0; c < 2; ++c) {  // scale (Q K^T . G), bf16, over K
    const int j0 = 64 * hf + 32 * c;
    float a[32];
    tmem_ld32(tl + j0, a);
    tmem_ld_wait();
#pragma unroll
    for (int jj = 0; jj < 32; ++jj) a[jj] = j0 + jj <= i ? p.scale * a[jj] * exp_diff(gi, gs[j0 + jj]) : 0.f;
#pragma unroll
    for (int c8 = 0; c8 < 4; ++c8)
      *reinterpret_cast<uint4*>(s + kOK + swz16(i, (j0 >> 3) + c8)) =
          make_uint4(pack_bf16x2(a[8 * c8], a[8 * c8 + 1]), pack_bf16x2(a[8 * c8 + 2], a[8 * c8 + 3]),
                     pack_bf16x2(a[8 * c8 + 4], a[8 * c8 + 5]), pack_bf16x2(a[8 * c8 + 6], a[8 * c8 + 7]));
  }
  fence_proxy_async_shared();
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    tc_fence_after();
    mma_tile(tmem + 256, sK, false, sE, true, false);
    umma_commit(bars + 1);
  }
  __syncwarp();
  wait_bar(bars + 1, 1, p.err);
  __syncwarp();
  tc_fence_after();
  const float fi = p.scale * exp_diff(gi, make_float2(0.f, 0.f));
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int j0 = 64 * hf + 32 * c;
    if (j0 >= p.dv) continue;
    float a[32], x[32];
    tmem_ld32(tl + 128 + j0, x);
    tmem_ld32(tl + 256 + j0, a);
    tmem_ld_wait();
    if (i < n) {
      uint4* og = reinterpret_cast<uint4*>(p.o + (row0 + i) * p.dv + j0);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 8 * v + 2 * e;
          w[e] = pack_bf16x2(fmaf(fi, x[j], a[j]), fmaf(fi, x[j + 1], a[j + 1]));
        }
        og[v] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct Plan {
  size_t W, U, K16, S, E, tab, amax, amax_bytes, total;
  int slots;
};
Plan plan_of(const GdrArgs& a) {
  Plan p{};
  const size_t slots = gdr_slots(a, kC), items = slots * a.H;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at = align_up(at + bytes, 1024);
    return x;
  };
  p.slots = (int)slots;
  p.W = take(items * 2 * kTile);
  p.U = take(items * kC * kC * 4);
  p.K16 = take(slots * a.Hk * kTile);
  p.S = take(items * kTile);
  p.E = take(items * kTile);
  p.tab = take(items * sizeof(Tables));
  p.amax_bytes = (size_t)gdr_sequences(a) * a.H * 4;
  p.amax = take(p.amax_bytes);
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

}  // namespace

bool gdr_tc_supported(const GdrArgs& a) {
  return a.io == LL_BF16 && a.dk >= 64 && a.dv >= 64 && a.T >= kGdrTcMinTokens;
}
size_t gdr_tc_fwd_workspace(const GdrArgs& a) { return plan_of(a).total; }

ll_status gdr_tc_fwd_launch(const GdrArgs& a) {
  const Plan pl = plan_of(a);
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
  p.log_alpha = a.log_alpha;
  p.beta = a.beta;
  p.state_in = a.state_in;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.state_out = a.state_out;
  p.W = ws + pl.W;
  p.U = reinterpret_cast<float*>(ws + pl.U);
  p.K16 = ws + pl.K16;
  p.S = ws + pl.S;
  p.E = ws + pl.E;
  p.tab = reinterpret_cast<Tables*>(ws + pl.tab);
  p.amax = reinterpret_cast<unsigned*>(ws + pl.amax);
  p.err = a.err;
  const int items = pl.slots * a.H, sms = sm_count(), slices = a.dv / kSlice;
  if (sms == 0) return LL_ERR_CUDA;
  LL_CUDA_OK(cudaFuncSetAttribute(gdr_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPrepSmem));
  LL_CUDA_OK(cudaFuncSetAttribute(gdr_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kScanSmem));
  LL_CUDA_OK(cudaFuncSetAttribute(gdr_out_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kOutSmem));
  LL_CUDA_OK(cudaMemsetAsync(p.amax, 0, pl.amax_bytes, a.stream));
  gdr_prep_kernel<<<std::min(items, sms), 256, kPrepSmem, a.stream>>>(p);
  LL_CUDA_OK(cudaGetLastError());
  gdr_scan_kernel<<<(unsigned)(gdr_sequences(a) * a.H * slices), 256, kScanSmem, a.stream>>>(p, slices);
  LL_CUDA_OK(cudaGetLastError());
  gdr_out_kernel<<<items, 256, kOutSmem, a.stream>>>(p);
  LL_CUDA_OK(cudaGetLastError());
  return LL_OK;
}

}  // namespace llattn

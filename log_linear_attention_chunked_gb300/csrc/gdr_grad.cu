// Gradient of the gated delta rule, the part that is parallel over chunks, in
// float32 on the CUDA cores (any io type and head sizes).
//
// For a chunk of C tokens let S0 be the state before it, D1 the adjoint of the
// state after it, e_t and w_t = A_t k_t the rows kept by the two recurrences,
// u = beta e, g the running log decay inside the chunk.  With
//   R_ij = scale exp(g_i - g_j) (do_i . u_j)     (j <= i)
//   N_ij = beta_i exp(g_i - g_j) (w_i . u_j)     (j <  i)
// the gradients are
//   dq = scale exp(g) (do S0) + R K
//   dk = R^T Q + exp(g_C - g) (u D1) - N^T K - N K - beta exp(g) (w S0)
//   dv = beta w,   dbeta = e . w
//   dlog_alpha_r = sum_{t >= r} (q_t . dq_t - v_t . dv_t) + <S1, D1>
// (q . dq is do . o, and do_t . o_t - u_t . w_t + beta_t w_t . (e_t - v_t) is
// the derivative by the running log decay at t), where
//   <S1, D1> = exp(g_C) <S0, D1> + sum_j exp(g_C - g_j) k_j . (u D1)_j.
// One CTA per (chunk, key head): the value heads that share it are taken in
// turn, so their dq and dk add up in registers in a fixed order.
#include "gdr.cuh"

namespace llattn {

namespace {

constexpr int kC = kGdrGradChunk;
constexpr int kThreads = 256;
constexpr int kLdC = kC + 1;

struct GradParams {
  GdrSeqs seqs;
  int dv;
  float scale;
  const void *q, *k, *v, *dout;
  const float *log_alpha, *beta, *states, *errors, *adjoints, *w;
  void *dq, *dkey, *dval;
  float *dlog_alpha, *dbeta;
};

inline size_t grad_smem(int dk, int dv) {
  return 4 * ((size_t)2 * kC * dk + (size_t)3 * kC * (dv + 1) + 2 * kC * kLdC + 8 * kC + 32);
}

// column j of thread tx (of 16) in a [.., DK] row: pieces of four side by side
template <int DK> __device__ __forceinline__ int col_of(int tx, int j) {
  if (DK >= 64) return (j >> 2) * 64 + tx * 4 + (j & 3);
  return tx * (DK / 16) + j;
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename IO, int DK>
__global__ void __launch_bounds__(kThreads) gdr_grad_kernel(GradParams p) {
  constexpr int NC = DK / 16;
  extern __shared__ float sm[];
  const int DV = p.dv, ldv = DV + 1;
  float* qs = sm;
  float* ks = qs + kC * DK;
  float* ds = ks + kC * DK;    // do
  float* es = ds + kC * ldv;   // e
  float* ws = es + kC * ldv;   // w
  float* R = ws + kC * ldv;
  float* N = R + kC * kLdC;
  float* ghi = N + kC * kLdC;  // running log decay, a pair
  float* glo = ghi + kC;
  float* into = glo + kC;      // exp(g_i)
  float* out = into + kC;      // exp(g_C - g_i)
  float* bs = out + kC;
  float* dg = bs + kC;
  float* kd = dg + kC;         // exp(g_C - g_j) k_j . (u D1)_j
  float* red = kd + kC;

  const int hk = blockIdx.x % p.seqs.Hk;
  const int slot = blockIdx.x / p.seqs.Hk;
  int seq, chunk;
  GdrSeq sq;
  if (!gdr_find(p.seqs, slot, kC, seq, chunk, sq)) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int t0 = chunk * kC, n = min(kC, sq.len - t0);
  const int G = p.seqs.H / p.seqs.Hk;
  const size_t krow0 = ((size_t)sq.row_b * p.seqs.Hk + hk) * p.seqs.T + sq.start + t0;

  for (int x = tid; x < kC * DK; x += kThreads) {
    const bool in = x / DK < n;
    qs[x] = in ? to_f(static_cast<const IO*>(p.q)[krow0 * DK + x]) : 0.f;
    ks[x] = in ? to_f(static_cast<const IO*>(p.k)[krow0 * DK + x]) : 0.f;
  }
  float aq[4][NC], ak[4][NC];  // dq and dk of this thread's rows, over the heads
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NC; ++j) aq[i][j] = ak[i][j] = 0.f;

  for (int hh = 0; hh < G; ++hh) {
    const int h = hk * G + hh;
    const size_t row0 = ((size_t)sq.row_b * p.seqs.H + h) * p.seqs.T + sq.start + t0;
    const size_t mat = ((size_t)slot * p.seqs.H + h) * DV * DK;
    const float* S0 = p.states + mat;
    const float* D1 = p.adjoints + mat;
    __syncthreads();  // the head before has read its rows
    for (int x = tid; x < kC * DV; x += kThreads) {
      const int t = x / DV, r = x - t * DV;
      const bool in = t < n;
      ds[t * ldv + r] = in ? to_f(static_cast<const IO*>(p.dout)[row0 * DV + x]) : 0.f;
      es[t * ldv + r] = in ? p.errors[row0 * DV + x] : 0.f;
      ws[t * ldv + r] = in ? p.w[row0 * DV + x] : 0.f;
    }
    if (tid < 32) {  // two tokens to a lane
      const int t = 2 * tid;
      const float2 x = make_float2(t < n ? gdr_log(p.log_alpha[row0 + t]) : 0.f, 0.f);
      const float2 y = make_float2(t + 1 < n ? gdr_log(p.log_alpha[row0 + t + 1]) : 0.f, 0.f);
      const float2 own = pair_add(x, y);
      float2 g = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float2 z = make_float2(__shfl_up_sync(0xffffffffu, g.x, o), __shfl_up_sync(0xffffffffu, g.y, o));
        if (tid >= o) g = pair_add(g, z);
      }
      float2 before = make_float2(__shfl_up_sync(0xffffffffu, g.x, 1), __shfl_up_sync(0xffffffffu, g.y, 1));
      if (tid == 0) before = make_float2(0.f, 0.f);
      before = pair_add(before, x);
      ghi[t] = before.x;
      glo[t] = before.y;
      ghi[t + 1] = g.x;
      glo[t + 1] = g.y;
    }
    if (tid < kC) bs[tid] = tid < n ? p.beta[row0 + tid] : 0.f;
    __syncthreads();
    if (tid < kC) {
      into[tid] = expf(ghi[tid] + glo[tid]);
      out[tid] = expf((ghi[kC - 1] - ghi[tid]) + (glo[kC - 1] - glo[tid]));
    }
    // ---- R and N
    {
      float r[4][4] = {}, m[4][4] = {};
#pragma unroll 4
      for (int d = 0; d < DV; ++d) {
        float ev[4], dv_[4], wv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) ev[j] = es[(tx + 16 * j) * ldv + d];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dv_[i] = ds[(4 * ty + i) * ldv + d];
          wv[i] = ws[(4 * ty + i) * ldv + d];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            r[i][j] = fmaf(dv_[i], ev[j], r[i][j]);
            m[i][j] = fmaf(wv[i], ev[j], m[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 4 * ty + i, col = tx + 16 * j;
          const float dec =
              col <= row ? bs[col] * expf((ghi[row] - ghi[col]) + (glo[row] - glo[col])) : 0.f;
          R[row * kLdC + col] = col <= row ? p.scale * dec * r[i][j] : 0.f;
          N[row * kLdC + col] = col < row ? bs[row] * dec * m[i][j] : 0.f;
        }
    }
    __syncthreads();
    // ---- do S0, w S0, e D1
    float x0[4][NC], x1[4][NC], x2[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NC; ++j) x0[i][j] = x1[i][j] = x2[i][j] = 0.f;
#pragma unroll 8
    for (int d = 0; d < DV; ++d) {  // (unrolled for the loads in flight)
      float sv[NC], av[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        sv[j] = S0[(size_t)d * DK + col_of<DK>(tx, j)];
        av[j] = D1[(size_t)d * DK + col_of<DK>(tx, j)];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = ds[(4 * ty + i) * ldv + d], w = ws[(4 * ty + i) * ldv + d], e = es[(4 * ty + i) * ldv + d];
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          x0[i][j] = fmaf(a, sv[j], x0[i][j]);
          x1[i][j] = fmaf(w, sv[j], x1[i][j]);
          x2[i][j] = fmaf(e, av[j], x2[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * ty + i;
      const float fq = p.scale * into[row], fw = -bs[row] * into[row], fe = bs[row] * out[row];
      float kdot = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        x2[i][j] *= fe;
        kdot = fmaf(x2[i][j], ks[row * DK + col_of<DK>(tx, j)], kdot);
        x0[i][j] *= fq;
        x1[i][j] = fmaf(fw, x1[i][j], x2[i][j]);
      }
      kdot = sum16(kdot);
      if (tx == 0) kd[row] = kdot;
    }
    // ---- R K, and R^T Q - (N + N^T) K
#pragma unroll 4
    for (int c = 0; c < kC; ++c) {
      float kv[NC], qv[NC];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        kv[j] = ks[c * DK + col_of<DK>(tx, j)];
        qv[j] = qs[c * DK + col_of<DK>(tx, j)];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * ty + i;
        const float a = R[row * kLdC + c], b = R[c * kLdC + row];
        const float m = -(N[row * kLdC + c] + N[c * kLdC + row]);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          x0[i][j] = fmaf(a, kv[j], x0[i][j]);
          x1[i][j] = fmaf(b, qv[j], fmaf(m, kv[j], x1[i][j]));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * ty + i;
      float qdot = 0.f, ew = 0.f, vw = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        qdot = fmaf(x0[i][j], qs[row * DK + col_of<DK>(tx, j)], qdot);
        aq[i][j] += x0[i][j];
        ak[i][j] += x1[i][j];
      }
      for (int d = tx; d < DV; d += 16) {
        const float w = ws[row * ldv + d];
        ew = fmaf(es[row * ldv + d], w, ew);
        if (row < n) {
          const size_t at = (row0 + row) * DV + d;
          const float g = bs[row] * w;
          vw = fmaf(to_f(static_cast<const IO*>(p.v)[at]), g, vw);
          static_cast<IO*>(p.dval)[at] = from_f<IO>(g);
        }
      }
      qdot = sum16(qdot);
      ew = sum16(ew);
      vw = sum16(vw);
      if (tx == 0) {
        dg[row] = qdot - vw;
        if (row < n) p.dbeta[row0 + row] = ew;
      }
    }
    // ---- <S1, D1>
    float dot = 0.f;
#pragma unroll 8
    for (int x = tid; x < DV * DK; x += kThreads) dot = fmaf(S0[x], D1[x], dot);
    dot = sum16(dot);
    if (tx == 0) red[ty] = dot;
    __syncthreads();
    if (tid < 32) {
      float2 sd = make_float2(tid < 16 ? red[tid] * into[kC - 1] : 0.f, 0.f);
      sd = pair_add(sd, make_float2(kd[2 * tid], 0.f));
      sd = pair_add(sd, make_float2(kd[2 * tid + 1], 0.f));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        sd = pair_add(sd, make_float2(__shfl_xor_sync(0xffffffffu, sd.x, o), __shfl_xor_sync(0xffffffffu, sd.y, o)));
      const float2 d1 = make_float2(dg[2 * tid + 1], 0.f);
      float2 g = pair_add(make_float2(dg[2 * tid], 0.f), d1);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float2 z = make_float2(__shfl_down_sync(0xffffffffu, g.x, o), __shfl_down_sync(0xffffffffu, g.y, o));
        if (tid + o < 32) g = pair_add(g, z);
      }
      float2 behind = make_float2(__shfl_down_sync(0xffffffffu, g.x, 1), __shfl_down_sync(0xffffffffu, g.y, 1));
      if (tid == 31) behind = make_float2(0.f, 0.f);
      behind = pair_add(behind, d1);
      const float2 at[2] = {pair_add(g, sd), pair_add(behind, sd)};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const size_t t = row0 + 2 * tid + e;
        if (2 * tid + e < n) p.dlog_alpha[t] = gdr_forgets(p.log_alpha[t]) ? 0.f : at[e].x;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * ty + i;
    if (row >= n) continue;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const size_t at = (krow0 + row) * DK + col_of<DK>(tx, j);
      static_cast<IO*>(p.dq)[at] = from_f<IO>(aq[i][j]);
      static_cast<IO*>(p.dkey)[at] = from_f<IO>(ak[i][j]);
    }
  }
}

template <typename IO, int DK>
ll_status run(const GradParams& p, unsigned grid, size_t smem, cudaStream_t st) {
  LL_CUDA_OK(cudaFuncSetAttribute(gdr_grad_kernel<IO, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)grad_smem(DK, 128)));
  gdr_grad_kernel<IO, DK><<<grid, kThreads, smem, st>>>(p);
  LL_CUDA_OK(cudaGetLastError());
  return LL_OK;
}
template <typename IO>
ll_status run_dk(int dk, const GradParams& p, unsigned grid, size_t smem, cudaStream_t st) {
  switch (dk) {
    case 16: return run<IO, 16>(p, grid, smem, st);
    case 32: return run<IO, 32>(p, grid, smem, st);
    case 64: return run<IO, 64>(p, grid, smem, st);
    case 128: return run<IO, 128>(p, grid, smem, st);
  }
  return LL_ERR_UNSUPPORTED;
}

struct RecPlan {
  size_t states, errors, adjoints, w, total;
};
RecPlan rec_plan(const GdrArgs& a) {
  RecPlan p{};
  const size_t mats = gdr_slots(a, kC) * a.H * a.dv * a.dk * 4, rows = (size_t)a.B * a.H * a.T * a.dv * 4;
  p.states = 0;
  p.adjoints = p.states + align_up(mats, 256);
  p.errors = p.adjoints + align_up(mats, 256);
  p.w = p.errors + align_up(rows, 256);
  p.total = p.w + align_up(rows, 256);
  return p;
}

}  // namespace

ll_status gdr_grad_launch(const GdrArgs& a, const float* states, const float* errors, const float* adjoints,
                          const float* w) {
  GradParams p{GdrSeqs{a.n_seqs ? a.seq_starts : nullptr, gdr_sequences(a), a.T, a.H, a.Hk},
               a.dv, a.scale, a.q, a.k, a.v, a.dout, a.log_alpha, a.beta, states, errors, adjoints, w,
               a.dq, a.dkey, a.dval, a.dlog_alpha, a.dbeta};
  const unsigned grid = (unsigned)(gdr_slots(a, kC) * a.Hk);
  const size_t smem = grad_smem(a.dk, a.dv);
  return a.io == LL_F32 ? run_dk<float>(a.dk, p, grid, smem, a.stream)
                        : run_dk<__nv_bfloat16>(a.dk, p, grid, smem, a.stream);
}

size_t gdr_fwd_workspace(const GdrArgs& a) { return gdr_tc_fwd_use(a) ? gdr_tc_fwd_workspace(a) : 0; }
int gdr_fwd_launches(const GdrArgs& a) { return gdr_tc_fwd_use(a) ? 3 : 1; }
ll_status gdr_fwd_launch(const GdrArgs& a) {
  return gdr_tc_fwd_use(a) ? gdr_tc_fwd_launch(a) : gdr_rec_fwd_launch(a);
}

size_t gdr_bwd_workspace(const GdrArgs& a) { return gdr_tc_bwd_use(a) ? gdr_tc_bwd_workspace(a) : rec_plan(a).total; }
int gdr_bwd_launches(const GdrArgs& a) { return gdr_tc_bwd_use(a) ? 4 : 2; }
ll_status gdr_bwd_launch(const GdrArgs& a) {
  if (gdr_tc_bwd_use(a)) return gdr_tc_bwd_launch(a);
  const RecPlan p = rec_plan(a);
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  float* states = reinterpret_cast<float*>(ws + p.states);
  float* adjoints = reinterpret_cast<float*>(ws + p.adjoints);
  float* errors = reinterpret_cast<float*>(ws + p.errors);
  float* w = reinterpret_cast<float*>(ws + p.w);
  ll_status st = gdr_rec_both_launch(a, states, errors, adjoints, w);
  if (st == LL_OK) st = gdr_grad_launch(a, states, errors, adjoints, w);
  return st;
}

}  // namespace llattn

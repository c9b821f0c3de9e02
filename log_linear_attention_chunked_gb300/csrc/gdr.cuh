// Gated delta rule (single state): shared declarations of its kernels.
//
//   S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   o_t = scale S_t q_t
// or, with e_t = v_t - alpha_t S_{t-1} k_t and u_t = beta_t e_t,
//   S_t = alpha_t S_{t-1} + u_t k_t^T.
//
// Sequences.  Unpacked, batch row b is one sequence of T tokens.  Packed
// (B == 1), sequence i is the tokens [starts[i], starts[i+1]) and has a state
// of its own.  Work on chunks of C tokens is dealt by slot: sequence i owns the
// slots base_i .. base_i + ceil(len_i / C) - 1 with base_i = floor(starts[i] / C)
// + i.  Since floor(a) + ceil(b) <= floor(a + b) + 1 these ranges never overlap
// and end below T / C + n, so no pass over the starts is needed to place them,
// and a slot finds its sequence by bisection.  A sequence whose bounds are not
// 0 <= start <= end <= T sets the device error word and is skipped.  Starts that are not
// ordered have at least one such; the others' slots may then overlap or go to another
// sequence, which spoils their results, but every slot stays below T / C + n and every
// chunk within its sequence's rows.
#pragma once

#include "common.cuh"

namespace llattn {

struct GdrArgs {
  int B, H, Hk, T, dk, dv, n_seqs;  // n_seqs = 0: unpacked
  ll_dtype io;
  float scale;
  const int32_t* seq_starts;
  const void *q, *k, *v;
  const float *log_alpha, *beta, *state_in;
  // forward
  void* o;
  float* state_out;
  // backward
  const void* dout;
  const float* dstate_out;
  void *dq, *dkey, *dval;
  float *dlog_alpha, *dbeta, *dstate_in;
  void* ws;
  size_t ws_bytes;
  cudaStream_t stream;
  unsigned* err;
};

inline int gdr_sequences(const GdrArgs& a) { return a.n_seqs ? a.n_seqs : a.B; }

struct GdrSeqs {
  const int32_t* starts;  // null: unpacked
  int n, T, H, Hk;
};

// Sequence `i`: its first row's index in [B, T] terms and its length (0 when
// its bounds are not valid).
struct GdrSeq {
  int row_b, start, len;
};
__device__ __forceinline__ bool gdr_seq(const GdrSeqs& s, int i, GdrSeq& r) {
  if (!s.starts) {
    r = GdrSeq{i, 0, s.T};
    return true;
  }
  const int a = s.starts[i], b = s.starts[i + 1];
  const bool ok = a >= 0 && a <= b && b <= s.T;
  r = GdrSeq{0, ok ? a : 0, ok ? b - a : 0};
  return ok;
}
// The sequence that a kernel with CTAs per sequence takes as its r-th (whole warps).  Up
// to 32 packed ones go from the longest down, so that a long one does not begin when the
// others are done (7 sequences, 448 CTAs: scans of 55 and 73 us became 53 and 71; a
// forward of 13, 832 CTAs, 234 us became 231).  Over many waves of CTAs they even out by
// themselves, and 0.8 us a CTA for the lengths cost more (17 sequences, 4352 CTAs: 205
// us became 227).
constexpr unsigned kGdrPickMost = 1216;  // eight CTAs to an SM
__device__ __forceinline__ int gdr_pick(const GdrSeqs& s, int r) {
  if (!s.starts || s.n > 32 || gridDim.x > kGdrPickMost) return r;
  const int lane = threadIdx.x & 31;
  GdrSeq q{0, 0, -1};
  if (lane < s.n) gdr_seq(s, lane, q);
  int rank = 0;
#pragma unroll 8
  for (int j = 0; j < 32; ++j) {
    const int l = __shfl_sync(0xffffffffu, q.len, j);
    rank += l > q.len || (l == q.len && j < lane);
  }
  return __ffs(__ballot_sync(0xffffffffu, rank == r)) - 1;
}
__device__ __forceinline__ int gdr_slot_base(const GdrSeqs& s, int i, int start, int C) {
  return s.starts ? start / C + i : i * ((s.T + C - 1) / C);
}
// The sequence and chunk of slot `c`; false when no valid chunk owns it.
__device__ __forceinline__ bool gdr_find(const GdrSeqs& s, int c, int C, int& seq, int& chunk, GdrSeq& r) {
  if (!s.starts) {
    const int per = (s.T + C - 1) / C;
    seq = c / per;
    chunk = c - seq * per;
    r = GdrSeq{seq, 0, s.T};
    return true;
  }
  int lo = 0, hi = s.n - 1;  // the last sequence with base <= c
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.starts[mid] / C + mid <= c) lo = mid;
    else hi = mid - 1;
  }
  seq = lo;
  if (!gdr_seq(s, seq, r)) return false;
  chunk = c - (r.start / C + seq);
  return chunk >= 0 && (long long)chunk * C < r.len;
}
inline size_t gdr_slots(const GdrArgs& a, int C) {
  return a.n_seqs ? (size_t)(a.T / C) + a.n_seqs : (size_t)a.B * ((a.T + C - 1) / C);
}

// log alpha below this is alpha = 0 in float32 either way; the bound keeps the
// running sums of a chunk finite for alpha = 0 (log alpha = -inf).
constexpr float kGdrMinLog = -1e4f;
__device__ __forceinline__ float gdr_log(float la) { return la < kGdrMinLog ? kGdrMinLog : la; }

// Is alpha zero in float32 (2^-149 is its smallest value)?  Then nothing depends on its
// logarithm, whose gradient the kernels otherwise have as a sum that ends in rounding.
__device__ __forceinline__ bool gdr_forgets(float la) { return la < -104.f; }

// exp of a log decay that a state is multiplied by again and again: near 1 expf's error,
// though within its bound, leans to one side and adds up; 1 + expm1f is off by its rounding.
__device__ __forceinline__ float gdr_alpha(float la) { return la > -0.5f ? 1.f + expm1f(la) : expf(la); }

// sums of floats as pairs (value and what its rounding left)
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
  const float s = a.x + b.x, t = s - a.x;
  const float e = (a.x - (s - t)) + (b.x - t) + (a.y + b.y);
  const float hi = s + e;
  return make_float2(hi, e - (hi - s));
}

// ---- launchers
size_t gdr_fwd_workspace(const GdrArgs& a);
ll_status gdr_fwd_launch(const GdrArgs& a);
int gdr_fwd_launches(const GdrArgs& a);
size_t gdr_bwd_workspace(const GdrArgs& a);
ll_status gdr_bwd_launch(const GdrArgs& a);
int gdr_bwd_launches(const GdrArgs& a);

// token by token, states in registers (gdr_rec.cu)
constexpr int kGdrGradChunk = 64;  // tokens between the states kept for the gradient
ll_status gdr_rec_fwd_launch(const GdrArgs& a);
ll_status gdr_rec_both_launch(const GdrArgs& a, float* kept_states, float* kept_errors, float* kept_adjoints,
                              float* kept_w);
ll_status gdr_grad_launch(const GdrArgs& a, const float* states, const float* errors, const float* adjoints,
                          const float* w);

// on the tensor cores (gdr_tc.cu), where its formats allow and its time is the shorter
bool gdr_tc_fwd_use(const GdrArgs& a);
bool gdr_tc_bwd_use(const GdrArgs& a);
size_t gdr_tc_fwd_workspace(const GdrArgs& a);
size_t gdr_tc_bwd_workspace(const GdrArgs& a);
ll_status gdr_tc_fwd_launch(const GdrArgs& a);
ll_status gdr_tc_bwd_launch(const GdrArgs& a);

ll_status gdr_decode_launch(int B, int H, int Hk, int dk, int dv, ll_dtype io, float scale, const int64_t* slots,
                            int n_slots, const void* q, const void* k, const void* v, const float* log_alpha,
                            const float* beta, float* states, void* o, cudaStream_t stream, unsigned* err);

}  // namespace llattn
